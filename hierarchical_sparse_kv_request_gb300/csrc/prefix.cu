// prefix.cu -- attention of a whole batch over a prefix that its requests share
// (include/hisparse_pages.h, hisparse_attend_prefix).
//
// The mathematics.  The heads of all requests are the rows of one matrix Q (M = R
// H rows of 576).  With s = scale * log2(e) * (q . row), a running reference m of
// the row maximum, l = sum 2^(s - m) and O = sum 2^(s - m) * latent over the rows
// seen so far; when s outgrows m by more than 8 (f16: see kBelowF16), m moves and l
// and O are multiplied by 2^(m_old - m_new).  A part comes in as one more row of score
// part_lse * log2(e) and value part.  out = O / l, lse = (m + log2 l) ln 2.
//
// Three launches.  expand_kernel reads the prefix's pages once and writes its rows
// to the workspace in 16 bits, in the layout that the tensor cores read, so that
// tiles come in as plain bulk copies whatever the format, the pages' size and the
// strides; rows that are not there are 0, and a bit a row says so.  prefix_kernel
// multiplies; its CTAs start beside expand_kernel's.  join_kernel adds up heads whose
// rows were split.
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
//   slots of 32 KB, two a tile (h = 0, 1), in a ring of five, of two parts: X_h are
//   values 128 h, Y_h values 256 + 128 h and on, of the CTA's own 64 keys.
//   After S the first CTA keeps X and gets, in Y, the other CTA's keys of its
//   values X; the second keeps Y and gets, in X, the first one's keys of Y.  A
//   descriptor is one for both CTAs: at X_h both have keys 0-63, at Y_h 64-127.
//   The rope part (8 KB) has a slot of its own.
// The queries do not fit either shared memory or what O and S leave of tensor
// memory (128 columns, S being there twice): 256 of their values are there, in both
// halves of the lanes, the other 320 in shared memory.
//   warps 0-3  softmax: a thread a lane, that is a head and half of the tile's keys;
//   warp 4     brings keys in, warp 5 the values of the other CTA's keys;
//   warp 6     of the first CTA issues the MMAs of S, up to two tiles ahead of warp 7,
//              which issues those of O; those of the second say what has come in there.
// The groups' tiles in a row are shared out among the pairs, wherever a group ends, so that
// each has as much to do, its groups' starts and ends counted.
//
// What bounds it.  With much to do, shared memory: a tile of 128 keys moves some 330 KB
// through each SM's (operands of S 112, of O 96, keys and values coming in 106, P 16) in
// 2,650 cycles, 125 of its 128 bytes a cycle, where the products alone take 2,184.  Without
// the copies a tile takes 2,330.  With little, a pair's start (1 thousand cycles, queries
// 4, while the rows are expanded) and end (5 to 7 for O, at some 25 bytes a cycle that an
// SM stores) and the launches around it.  Measured on GB300, GPU time of a call: 256
// requests of 16 heads over 40,000 rows 228 us (1,564 TFLOP/s, 0.84 of cuBLAS's best), 241
// in a long row of calls (1,479, 0.87 of its sustained rate: the power limit takes the clock
// down); 32 of 128 heads over 8,192 62; 32 of 16 over 8,192 22.3; 37 of 40 over 5,003 27.7;
// 4 of 16 over 2,048 11.
// Rounding.  Queries are exact (see ScoreFactors), and latent values of 4-bit rows, and of
// 8-bit rows with powers of two as scales, too, in f16 as far as they are among its normal
// numbers.  P is rounded to the model's type (half a step: 2^-8 of a probability in bf16),
// which the product's two operands share, and their sum l is of the unrounded ones, so that
// lse does not feel it: out's error against 64 bits is 1.7 to 2.0 x 10^-3 in bf16 (the
// plain 32-bit form's: 1.65) and 2.5 x 10^-4 in f16 (2.1).  Scores, references, sums and
// O are 32-bit, and sums add up a tile at a time.
#include <atomic>

#include "pages.cuh"

namespace hs {
namespace {

constexpr int PAIR_HEADS = 128, CTA_HEADS = 64, KEYS = 128;
constexpr int MAX_PAIRS = 76;                    // pairs of SMs of a GB300 (with fewer, in waves)
constexpr uint32_t BLOCK = 64 * 128;             // 64 values of 64 keys, swizzled
constexpr uint32_t PART = 2 * BLOCK, SLOT = 2 * PART;
constexpr uint32_t HALF_TILE = 9 * BLOCK;        // 64 keys: X0 Y0 X1 Y1 rope, as they go into the slots
constexpr uint32_t TILE_BYTES = 2 * HALF_TILE;
constexpr int SLOTS = 5;
constexpr int Q_TMEM = 4, Q_SMEM = 9 - Q_TMEM;   // blocks of the queries

constexpr uint32_t ROPE_AT = SLOTS * SLOT, Q_AT = ROPE_AT + BLOCK, P_AT = Q_AT + Q_SMEM * BLOCK;
constexpr uint32_t MISC_AT = P_AT + 2 * BLOCK;
constexpr int PX_NT = 256, SOFTMAX = 4, KEY_WARP = 4, VALUE_WARP = 5, MMA_WARP = 6;

// columns of tensor memory
constexpr uint32_t T_O = 0, T_S = 256, T_Q = 384;      // (S of two tiles)

struct PrefixSmem {
    uint64_t keys[SLOTS], rope, values[2];              // arrived (in the first CTA: in both)
    uint64_t slot_free[SLOTS];                          // the products that read it are done
    uint64_t scored[2], added;                          // S is there; O is
    uint64_t queries, read[2], weighed;                 // (in the first CTA, from both) Q is there, S read, P there
    uint64_t drained[2];
    uint32_t tmem;
    int gave_up;
    float top[2][2][CTA_HEADS];      // [tile % 2][half of the keys]
    float sum[2][CTA_HEADS];
};
constexpr size_t PX_SMEM = MISC_AT + sizeof(PrefixSmem);
static_assert(PX_SMEM <= 232448, "shared memory of a CTA");

// The latent block (of 64 values; 8: the rope part) at place n of a half tile.
__host__ __device__ constexpr int block_at(int n) { return n == 8 ? 8 : (n >> 2) * 2 + (n >> 1 & 1) * 4 + (n & 1); }

// How a call is cut up, and its workspace.  Pair p has the tiles from start[p] to
// start[p + 1], in the order of groups and tiles.
struct PrefixParts {
    int tiles;               // of 128 keys
    int groups;              // of 128 heads
    int pairs;
    int joins;               // groups that several pairs have some of
    struct Place {
        int32_t group, tile;
    } start[MAX_PAIRS + 1];
    // pair `first` has the group's first tile, the parts - 1 that follow begin in the middle
    // of it
    struct Join {
        int32_t group;
        int16_t first, parts;
    } join[MAX_PAIRS];
    uint8_t *image;          // [tiles][2] half tiles
    uint8_t *there;          // [tiles][32] the low four bits: a bit a key
    uint8_t *o;              // [pairs][2] parts of O of 128 heads that a pair does not have whole (see
                             // part_at): of a group that it begins in the middle, of one from its start
    float2 *ml;              // [pairs][2][128] reference and sum
};

// A part of O: per CTA and warp of 32 heads by 256 values, 8 images of 32 values, the
// 16-byte units of a head's 128 bytes swizzled.  Where values 4 n to 4 n + 3 of head i
// of the pair's 128 are.
constexpr int PART_IMAGE = 32 * 128;
__host__ __device__ __forceinline__ int part_at(int i, int n)
{
    const int warp = (i >> 6) * 4 + (n >> 6) * 2 + (i >> 5 & 1), h = i & 31;
    return (warp * 8 + (n >> 3 & 7)) * PART_IMAGE + h * 128 + (((n ^ h) & 7) << 4);
}

// ---- expand ------------------------------------------------------------------------

// Warps without a word to each other: a round of EX_ROWS rows, a byte of `there`, or, with
// ROUNDS 2, another behind it, whose rows are called into L2 meanwhile.  64 registers, 7
// warps and no shared memory: a CTA finds a place beside prefix_kernel's (192 registers,
// and nearly all shared memory), which so has its tensor memory and its queries, 3 to 4 us,
// by when the rows are there.
constexpr int EX_NT = 224, EX_ROWS = 4;

template <int DT, int ROW, int ROUNDS>
__global__ void __maxnreg__(64) expand_kernel(const __grid_constant__ PrefixLaunch a, const __grid_constant__ PrefixParts w)
{
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) * gridDim.x + blockIdx.x, warps = EX_NT / 32 * gridDim.x;
    const int rounds = w.tiles * (KEYS / EX_ROWS);
    after_launch_before();
    // prefix_kernel may be placed now: after this wait, as it reads its queries ahead of
    // its own
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int ahead = lane / EX_ROWS, t = (warp + ahead * warps) * EX_ROWS + lane % EX_ROWS;
    const uint8_t *mine = nullptr;
    bool bad = false;
    if (ahead < ROUNDS && t < a.len) {
        const int b = t / a.bs;
        const int32_t page = a.table[b];
        const int64_t row = (int64_t)page * a.bs + (t - b * a.bs);
        if (page >= 0 && row < a.num_rows)
            mine = a.rows + row * a.row_stride;
        else
            bad = page != -1;
    }
    if (ROUNDS > 1 && ahead == 1 && mine)      // (into L2)
#pragma unroll
        for (int x = 0; x < ROW; x += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(mine + x));
    const uint32_t named = __ballot_sync(0xffffffffu, mine != nullptr);
#pragma unroll 1
    for (int k = 0; k < ROUNDS && warp + k * warps < rounds; ++k) {
        const int n = warp + k * warps;
        Latent8<ROW> v[EX_ROWS][2];
        uint4 rope[EX_ROWS];
#pragma unroll
        for (int j = 0; j < EX_ROWS; ++j) {
            const uint8_t *p = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), k * EX_ROWS + j));
            rope[j] = make_uint4(0, 0, 0, 0);
            if (p) {
                v[j][0].fetch(p, lane);
                v[j][1].fetch(p, lane + 32);
                if (lane < 8) rope[j] = ld_dev_v4(p + rope_at(ROW) + lane * 16);
            }
        }
        if (lane == 0) w.there[n] = (uint8_t)(named >> (k * EX_ROWS) & ((1u << EX_ROWS) - 1));
        uint8_t *half = w.image + (int64_t)(n / (64 / EX_ROWS)) * HALF_TILE;
#pragma unroll
        for (int j = 0; j < EX_ROWS; ++j) {
            const int i = n % (64 / EX_ROWS) * EX_ROWS + j;
            const uint32_t x = ((lane & 7) ^ (i & 7)) << 4;
            // unit lane + 32 k is in block lane / 8 + 4 k, which is at place 0 1 4 5, 2 3 6 7
            const int place = (lane >> 4) * 4 + (lane >> 3 & 1);
            st_v4(half + place * BLOCK + i * 128 + x, latent8<DT, ROW>(v[j][0]));
            st_v4(half + (place + 2) * BLOCK + i * 128 + x, latent8<DT, ROW>(v[j][1]));
            if (lane < 8) st_v4(half + 8 * BLOCK + i * 128 + x, rope[j]);
        }
    }
    if (__any_sync(0xffffffffu, bad) && a.status)
        for (int r = lane; r < a.R; r += 32) record_status(a.status, r, kStatusBadResident);
}

// ---- pairs of CTAs ---------------------------------------------------------------

// In any CTA of the cluster.  (Releases to the thread's own CTA: what the other's
// tensor core reads is in that CTA's shared and tensor memory.  A release to the
// cluster takes 900 cycles.)
__device__ __forceinline__ void arrive_in(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
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

// The mbarrier expects the bytes already.
__device__ __forceinline__ void bring(uint32_t dst, const uint8_t *src, uint32_t bytes, uint32_t bar)
{
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

// The bits of 32 keys, four a byte.
__device__ __forceinline__ uint32_t bits_of(uint32_t x, uint32_t y)
{
    auto half = [](uint32_t z) {
        z = (z | z >> 4) & 0x00FF00FFu;
        return (z | z >> 8) & 0xFFFFu;
    };
    return half(x) | half(y) << 16;
}

// A CTA's heads of a group: all 64 but of the last, of which both have half, so that
// neither brings in, keeps up and stores more than it must.
__host__ __device__ __forceinline__ int heads_of_cta(int heads, int group)
{
    const int left = heads - group * PAIR_HEADS;
    return left < PAIR_HEADS ? (left + 1) / 2 : CTA_HEADS;
}

// A head's request and number.  (At most 2^13 requests of 2^10 heads.)
struct HeadPlace {
    int r, h;
    __device__ __forceinline__ HeadPlace(const PrefixLaunch &a, int head) : r(head / a.H), h(head - r * a.H) {}
};

// How scores are made: queries (two a word) are multiplied by `query`, the products by f,
// positive, and `more`, which makes base-2 scores.  The sign of the scale goes into the
// queries, and in bf16, which has the range for it, its power of two: a product is then
// about as large as the score, and beyond 32 bits only if that is.  (A query times a power
// of two is exact from 2^-126 on.)  In f16 products are far within 32 bits, and a factor of
// 4 comes off f where log2(e) would take it beyond them.
template <int DT>
struct ScoreFactors {
    uint32_t query;
    float f, more;
    __device__ __forceinline__ explicit ScoreFactors(float scale)
    {
        const float size = fabsf(scale);
        uint32_t by;
        more = 1.0f;
        if (!(size <= FLT_MAX)) {
            by = 0x7FFFu;      // NaN
            f = 1.0f;
        } else if (size == 0.0f) {
            by = 0u;           // (f 0 would make NaN of the -inf of a row that is not there)
            f = 1.0f;
        } else if (DT == kBf16) {
            const uint32_t bits = __float_as_uint(size), e = max(bits >> 23, 1u);
            by = e << 7;
            f = (bits >> 23 ? __uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u) : size * 0x1p126f) * kLog2e;
        } else {
            by = 0x3C00u;
            if (size > 0x1p126f) more = 4.0f;
            f = size * (kLog2e / more);
        }
        if (scale < 0.0f) by |= 0x8000u;
        query = by * 0x10001u;
    }
    __device__ __forceinline__ uint32_t of(uint32_t x) const
    {
        uint32_t y;
        if (DT == kBf16)
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(query));
        else
            asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(query));
        return y;
    }
};

// A reference is a rounded score, and the weights' exponents are differences from it that
// leave that rounding out: half a step, from here on a sixteenth and more (at 2^29 a factor
// of 2^32, at 2^31 beyond 32 bits).  Scores are then rounded too before the reference comes
// off.  (In a branch of its own, as far as P's stores: with the exponents chosen in the
// loop that all tiles go through 32 x 128 heads over 8,192 rows take 63.0 us instead of 62.0,
// 61.6 with no such branch.)
constexpr float kFarReference = 1 << 20;

// In f16 weights below 2^-14 lose bits and those below 2^-25 are 0, however many they are: the
// reference lies 2^7 below the largest score when it moves, and moves for one above 2^15 of it
// (65,504 is f16's largest; a far reference, rounded to more than that, stays where the score
// is, as its neighbours weigh nothing).  So at most 2^-32 of the largest weight is lost a
// row, 2^-12 with the most rows, half of out's own half step.  (With 2^9 the reference moves
// more often: 32 x 128 heads over 8,192 rows 63.3 us, 37 x 40 over 5,003 28.2; 2^7 62.4 and 27.8, as
// with the reference at the largest score.)
constexpr float kBelowF16 = 7.0f, kAboveF16 = 15.0f;

// Whether all threads that meet at a named barrier go on.  (Nothing limits this
// wait: all of them come here, whatever has gone wrong.)
__device__ __forceinline__ bool meet(int id, int threads, bool go)
{
    uint32_t all;
    asm volatile("{\n"
                 ".reg .pred p, q;\n"
                 "setp.ne.u32 p, %1, 0;\n"
                 "barrier.cta.red.and.pred q, %2, %3, p;\n"
                 "selp.u32 %0, 1, 0, q;\n"
                 "}"
                 : "=r"(all)
                 : "r"((uint32_t)go), "r"(id), "r"(threads)
                 : "memory");
    return all != 0;
}

template <int DT>
__global__ void __cluster_dims__(2, 1, 1) __maxnreg__(192)
    prefix_kernel(const __grid_constant__ PrefixLaunch a, const __grid_constant__ PrefixParts w)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    PrefixSmem &sm = *reinterpret_cast<PrefixSmem *>(smem + MISC_AT);
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1;
    const PrefixParts::Place begin = w.start[pair], end = w.start[pair + 1];
    // tiles of this pair, over all its groups of heads
    const int count = (end.group - begin.group) * w.tiles + end.tile - begin.tile;
    auto bar = [](const uint64_t &b) { return smem_u32(&b); };

    if (warp == MMA_WARP) {
        if (lane == 0) {
            const int both = rank == 0 ? 2 : 1;      // the first CTA also hears of the second
            for (int s = 0; s < SLOTS; ++s) mbar_init(bar(sm.keys[s]), both), mbar_init(bar(sm.slot_free[s]), 1);
            mbar_init(bar(sm.rope), both);
            for (int s = 0; s < 2; ++s) {
                mbar_init(bar(sm.values[s]), both);
                mbar_init(bar(sm.scored[s]), 1);
                mbar_init(bar(sm.read[s]), 2 * SOFTMAX);
            }
            mbar_init(bar(sm.added), 1);
            mbar_init(bar(sm.queries), 2 * SOFTMAX);
            mbar_init(bar(sm.weighed), 2 * SOFTMAX);
            mbar_init(bar(sm.drained[0]), 1);
            mbar_init(bar(sm.drained[1]), 1);
            sm.gave_up = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    volatile int *gave_up = &sm.gave_up;
    auto all = [](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
    bool ok = true;
    cluster_wait();      // the other CTA's mbarriers are there, and its tensor memory
    // (the softmax warps read the queries ahead of this wait: see expand_kernel)
    if (warp >= SOFTMAX) after_launch_before();
    // join_kernel may be placed now, as it waits before it does anything.  (Not so the
    // caller's next launch, where no join follows: see hisparse_set_programmatic_launch.)
    if (w.joins > 0 && warp == MMA_WARP) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp < SOFTMAX) {
        // ---- softmax: a thread has head (warp % 2) 32 + lane of the CTA's, and half of
        // the keys, and in the end half of the values -----------------------------------
        const int i = (warp & 1) * 32 + lane, half = warp >> 1;
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        const uint32_t queries_at = in_cta(bar(sm.queries), 0), read_at = in_cta(bar(sm.read[0]), 0), weighed_at = in_cta(bar(sm.weighed), 0);
        auto tell = [&](uint32_t at) {
            __syncwarp();
            if (lane == 0) arrive_in(at);
        };
        auto meet_half = [&](bool go) { return meet(1 + (warp & 1), 64, go); };      // the warp with the heads' other half
        auto meet_all = [&](bool go) { return meet(3, SOFTMAX * 32, go); };
        constexpr float BELOW = DT == kF16 ? kBelowF16 : 0.0f, ABOVE = DT == kF16 ? kAboveF16 : kMoveAbove;
        const ScoreFactors<DT> factors(a.scale);
        const float f = factors.f;
        // The queries of a group, times their factor: eight threads a head's 128 bytes, all
        // of it on its way at once; then through P's place, 16 KB at a time, to a thread's
        // lane.  (A thread its own head's, 16 bytes of 32 heads a load: 11 thousand cycles
        // against 5.)
        const int heads = a.R * a.H;
        auto place_queries = [&](int group) {
            const int share = heads_of_cta(heads, group), head0 = group * PAIR_HEADS + rank * share;
            const int unit = lane & 7, first = warp * 4 + (lane >> 3);      // heads first + 16 k
            uint4 v[9][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int head = head0 + first + 16 * k;
                const bool on = first + 16 * k < share && head < heads;
                const HeadPlace at(a, on ? head : 0);
                const uint8_t *q = a.q + at.r * a.q_rs + at.h * a.q_hs + unit * 16;
#pragma unroll
                for (int b = 0; b < 9; ++b) {
                    v[b][k] = make_uint4(0, 0, 0, 0);
                    if (on) v[b][k] = ld_dev_v4(q + block_at(b) * 128);
                }
            }
            auto put = [&](uint32_t block, const uint4 (&x)[4]) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int h = first + 16 * k;
                    st_smem_v4(block + h * 128 + ((unit ^ (h & 7)) << 4),
                               make_uint4(factors.of(x[k].x), factors.of(x[k].y), factors.of(x[k].z), factors.of(x[k].w)));
                }
            };
#pragma unroll
            for (int b = 0; b < Q_SMEM; ++b) put(base + Q_AT + b * BLOCK, v[Q_TMEM + b]);
#pragma unroll
            for (int b = 0; b < Q_TMEM; b += 2) {
                put(base + P_AT, v[b]);
                put(base + P_AT + BLOCK, v[b + 1]);
                meet_all(true);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t y[32];
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const uint4 z = ld_smem_v4(base + P_AT + k * BLOCK + i * 128 + ((x ^ (i & 7)) << 4));
                        y[4 * x] = z.x, y[4 * x + 1] = z.y, y[4 * x + 2] = z.z, y[4 * x + 3] = z.w;
                    }
                    tmem_st_32(lanes + T_Q + (b + k) * 32, y);
                }
                meet_all(true);
            }
            tmem_wait_st();
            fence_async_smem();
            tc_fence_before();
            tell(queries_at);
        };
        // O of the warp's 32 heads, 32 columns from c on at a time, so that eight threads
        // have 128 bytes of a head: take(c, k, the four at columns c + 4 (lane % 8) of
        // head 4 k + lane / 8).  By way of the warp's quarter of P's place.
        const uint32_t stage = base + P_AT + warp * 4096;
        auto all_columns = [&](auto take) {
            uint32_t o[32];
            tmem_ld_32(lanes + T_O, o);
#pragma unroll 1
            for (int c = 0; c < 256; c += 32) {
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    st_smem_v4(stage + lane * 128 + ((x ^ (lane & 7)) << 4), make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]));
                if (c < 224) tmem_ld_32(lanes + T_O + c + 32, o);
                __syncwarp();
                uint4 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int h = k * 4 + (lane >> 3);
                    v[k] = ld_smem_v4(stage + h * 128 + (((lane & 7) ^ (h & 7)) << 4));
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) take(c, k, v[k]);
            }
        };
        int n = 0;
        const int last_group = end.tile > 0 ? end.group : end.group - 1;
        for (int group = begin.group, t0 = begin.tile; group <= last_group; ++group, t0 = 0) {
            // (all four warps come here as often, whatever has gone wrong; P's place is free)
            if (!(ok = meet_all(ok))) break;
            const int t1 = group == end.group ? end.tile : w.tiles;
            const int share = heads_of_cta(heads, group), head = group * PAIR_HEADS + rank * share + i;
            const bool on = i < share && head < heads;
            const int here = __popc(__ballot_sync(0xffffffffu, on));      // of the warp's heads
            place_queries(group);
            if (group == begin.group) after_launch_before();
            float m = -INFINITY, l = 0.0f;
            bool far = factors.more != 1.0f;      // or one of the warp's references is: see kFarReference
            const uint8_t *there = w.there + half * 16;
            uint4 next = *reinterpret_cast<const uint4 *>(there + (int64_t)t0 * 32);
            for (int t = t0; t < t1; ++t, ++n) {
                const uint4 named = next;
                if (t + 1 < t1) next = *reinterpret_cast<const uint4 *>(there + (int64_t)(t + 1) * 32);
                ok = ok && all(mbar_wait(bar(sm.scored[n & 1]), (n >> 1) & 1, gave_up));
                tc_fence_after();
                uint32_t v[2][32];
                tmem_ld_32(lanes + T_S + (n & 1) * 64, v[0]);
                tmem_ld_32(lanes + T_S + (n & 1) * 64 + 32, v[1]);
                tmem_wait_ld();
                tc_fence_before();
                tell(read_at + (n & 1) * 8);
                float (&x)[2][32] = reinterpret_cast<float (&)[2][32]>(v);
                if ((named.x & named.y & named.z & named.w) != 0x0F0F0F0Fu) {
                    const uint32_t lo = bits_of(named.x, named.y), hi = bits_of(named.z, named.w);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (!(lo >> j & 1u)) x[0][j] = -INFINITY;
                        if (!(hi >> j & 1u)) x[1][j] = -INFINITY;
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
                float s = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * f * factors.more;
                sm.top[n & 1][half][i] = s;
                if (!(ok = meet_half(ok))) break;
                s = fmaxf(s, sm.top[n & 1][half ^ 1][i]);
                // P and O are free once the product before is done: O times d, and P in its place
                auto add = [&](bool is_free, bool moves, float d) {
                    if (!all(is_free) && !(ok = all(mbar_wait(bar(sm.added), (n - 1) & 1, gave_up)))) return;
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
                        for (int y = 0; y < 4; ++y)
                            st_smem_v4(p_at + (((k * 4 + y) ^ (i & 7)) << 4),
                                       make_uint4(v[k][4 * y], v[k][4 * y + 1], v[k][4 * y + 2], v[k][4 * y + 3]));
                    fence_async_smem();
                    tc_fence_before();
                    tell(weighed_at);
                };
                float d = 1.0f;
                // (the difference: m + ABOVE may round to the next number)
                const bool moves = __any_sync(0xffffffffu, s - m > ABOVE || far);
                if (moves) {
                    const float to = fmaxf(m, fabsf(s) < kFarReference ? s - BELOW : s);
                    d = to == -INFINITY ? 1.0f : ex2(m - to);
                    m = to;
                    l *= d;
                    far = factors.more != 1.0f || __any_sync(0xffffffffu, fabsf(m) >= kFarReference && m != -INFINITY);
                    if (far) {
                        const float r = m == -INFINITY ? 0.0f : -m;
                        auto weight = [&](float product) { return ex2(fmaf(__fmul_rn(product, f), factors.more, r)); };
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int j = 0; j < 32; j += 2) {
                                const float p0 = weight(x[k][j]), p1 = weight(x[k][j + 1]);
                                l += p0 + p1;
                                v[k][j >> 1] = floats_to_pair<DT>(p0, p1);
                            }
                        add(n == 0, true, d);
                        continue;
                    }
                }
                // (asked ahead of the exponentials, which hide how long that takes)
                const bool is_free = n == 0 || mbar_try(bar(sm.added), (n - 1) & 1);
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
                add(is_free, moves, d);
            }
            ok = ok && all(mbar_wait(bar(sm.added), (n - 1) & 1, gave_up));
            tc_fence_after();
            const float part_lse = a.part && on ? a.part_lse[head] : -INFINITY;      // (lse may be the same)
            sm.sum[half][i] = l;
            if (!(ok = meet_half(ok))) continue;      // (to the barrier of all)
            l += sm.sum[half ^ 1][i];
            meet_half(true);
            if (t0 == 0 && t1 == w.tiles) {      // all of the heads' rows: out
                const HeadPlace at(a, on ? head : 0);
                float weight = 0.0f, scale = 1.0f;
                const uint8_t *part = nullptr;
                if (a.part) {
                    scale = add_part(m, l, part_lse, &weight);
                    if (weight != 0.0f) part = a.part + at.r * a.part_rs + at.h * a.part_hs + half * 512;
                }
                const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
                if (on && half == 0 && a.lse) a.lse[head] = log2_sum(m, l) * kLn2;
                scale *= inv;
                weight *= inv;
                const unsigned long long to = reinterpret_cast<unsigned long long>(on ? a.out + at.r * a.out_rs + at.h * a.out_hs + half * 512 : nullptr);
                const unsigned long long from = reinterpret_cast<unsigned long long>(part);
                if (here > 0) all_columns([&](int c, int k, uint4 o) {
                    const int h = k * 4 + (lane >> 3);
                    const float fo = __shfl_sync(0xffffffffu, scale, h), fp = __shfl_sync(0xffffffffu, weight, h);
                    uint8_t *dst = reinterpret_cast<uint8_t *>(__shfl_sync(0xffffffffu, to, h));
                    const uint8_t *src = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, from, h));
                    if (!dst) return;
                    const int64_t off = c * 2 + (lane & 7) * 8;
                    float2 x = make_float2(__uint_as_float(o.x) * fo, __uint_as_float(o.y) * fo);
                    float2 y = make_float2(__uint_as_float(o.z) * fo, __uint_as_float(o.w) * fo);
                    if (src) {
                        const uint2 p = *reinterpret_cast<const uint2 *>(src + off);
                        const float2 px = pair_to_float<DT>(p.x), py = pair_to_float<DT>(p.y);
                        x = make_float2(fmaf(px.x, fp, x.x), fmaf(px.y, fp, x.y));
                        y = make_float2(fmaf(py.x, fp, y.x), fmaf(py.y, fp, y.y));
                    }
                    *reinterpret_cast<uint2 *>(dst + off) = make_uint2(floats_to_pair<DT>(x.x, x.y), floats_to_pair<DT>(y.x, y.y));
                });
            } else {
                // As images of 32 columns of the warp's 32 heads (see part_at), by bulk copies:
                // an SM's own stores take twice as long.  In P's place and, for the others to
                // go out meanwhile, in the queries', which no product reads any more.
                const int64_t place = (int64_t)pair * 2 + (t0 == 0);
                if (half == 0) w.ml[place * PAIR_HEADS + rank * CTA_HEADS + i] = make_float2(m, l);
                uint8_t *to = w.o + (place * 8 + rank * 4 + warp) * (8 * PART_IMAGE);
                uint32_t o[32];
                tmem_ld_32(lanes + T_O, o);
#pragma unroll 1
                for (int c = 0; here > 0 && c < 8; ++c) {
                    const uint32_t image = c % 3 == 2 ? base + P_AT + warp * PART_IMAGE : base + Q_AT + (warp * 2 + c % 3) * PART_IMAGE;
                    if (c >= 3) asm volatile("cp.async.bulk.wait_group.read 2;" ::: "memory");      // (lane 0's)
                    __syncwarp();
                    tmem_wait_ld();
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        st_smem_v4(image + lane * 128 + ((x ^ (lane & 7)) << 4), make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]));
                    if (c < 7) tmem_ld_32(lanes + T_O + (c + 1) * 32, o);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n"
                                     "cp.async.bulk.commit_group;" ::"l"(to + c * PART_IMAGE),
                                     "r"(image), "r"(here * 128)
                                     : "memory");
                }
                asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
            }
            tc_fence_before();
        }
    } else if (warp == KEY_WARP) {
        // ---- this CTA's keys of every tile ------------------------------------------
        int slot = 0, tile = begin.tile;
        uint32_t slot_phase = 1;      // (nothing to wait for the first time round)
        for (int n = 0; ok && n < count; ++n) {
            const uint8_t *src = w.image + ((int64_t)tile * 2 + rank) * HALF_TILE;
            for (int h = 0; h < 2; ++h) {
                if (!(ok = ok && all(mbar_wait(bar(sm.slot_free[slot]), slot_phase, gave_up)))) break;
                if (elect_one()) {
                    const uint32_t here = bar(sm.keys[slot]);
                    mbar_expect(here, SLOT);
                    bring(base + slot * SLOT, src + h * SLOT, SLOT, here);
                }
                __syncwarp();
                if (++slot == SLOTS) slot = 0, slot_phase ^= 1;
            }
            if (++tile == w.tiles) tile = 0;
        }
    } else if (warp == VALUE_WARP) {
        // ---- the other CTA's keys, for this one's values --------------------------------
        int slot = 0, tile = begin.tile;
        const uint32_t to = rank == 0 ? PART : 0;      // Y or X
        auto rope = [&](int tile) {
            if (elect_one()) {
                mbar_expect(bar(sm.rope), BLOCK);
                bring(base + ROPE_AT, w.image + ((int64_t)tile * 2 + rank) * HALF_TILE + 2 * SLOT, BLOCK, bar(sm.rope));
            }
            __syncwarp();
        };
        rope(tile);
        for (int n = 0; ok && n < count; ++n) {
            if (!(ok = all(mbar_wait(bar(sm.scored[n & 1]), (n >> 1) & 1, gave_up)))) break;
            const uint8_t *src = w.image + ((int64_t)tile * 2 + (rank ^ 1)) * HALF_TILE + rank * PART;
            if (elect_one()) {
                const uint32_t here = bar(sm.values[n & 1]);
                mbar_expect(here, 2 * PART);
                for (int h = 0; h < 2; ++h) {
                    const int s = slot + h < SLOTS ? slot + h : 0;
                    bring(base + s * SLOT + to, src + h * SLOT, PART, here);
                }
            }
            __syncwarp();
            slot += 2;
            if (slot >= SLOTS) slot -= SLOTS;
            if (++tile == w.tiles) tile = 0;
            if (n + 1 < count) rope(tile);
        }
    } else if (rank == 1) {
        // ---- what has come in here, to the first CTA --------------------------------------
        auto tell = [&](const uint64_t &b, uint32_t phase) {
            ok = ok && all(mbar_wait(bar(b), phase, gave_up));
            if (ok && lane == 0) arrive_in(in_cta(bar(b), 0));
        };
        int slot = 0;
        uint32_t slot_phase = 0;
        for (int n = 0; ok && n < count; ++n) {
            if (warp == MMA_WARP) {
                for (int h = 0; h < 2; ++h) {
                    tell(sm.keys[slot], slot_phase);
                    if (++slot == SLOTS) slot = 0, slot_phase ^= 1;
                }
                tell(sm.rope, n & 1);
            } else {
                tell(sm.values[n & 1], (n >> 1) & 1);
            }
        }
    } else if (elect_one()) {
        // ---- MMA issue, of S and of O by one thread each, from its first wait to its last
        // (leaving and entering an elected thread's part around each wait cost 300 cycles),
        // in short loops.  A thread's waits, and the fences behind them, take some hundred
        // cycles, in which the other's MMAs go on. -----------------------------------------
        auto wait = [&](const uint64_t &b, uint32_t phase) { return ok = ok && mbar_wait(bar(b), phase, gave_up); };
        int slot = 0, tile = begin.tile;
        bool begins = true;      // a group of heads
        if (warp == MMA_WARP) {
            constexpr uint32_t qk = mma_desc(128, KEYS, DT == kBf16, false);
            int group = 0;
            uint32_t slot_phase = 0;
            auto next_slot = [&]() {
                const uint64_t k_desc = smem_desc(base + slot * SLOT, 16, 1024);
                if (++slot == SLOTS) slot = 0, slot_phase ^= 1;
                return k_desc;
            };
#pragma unroll 1
            for (int n = 0; ok && n < count; ++n) {
                wait(sm.keys[slot], slot_phase);
                if (begins) wait(sm.queries, group++ & 1);
                if (n > 1) wait(sm.read[n & 1], ((n >> 1) - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + T_S + (n & 1) * 64;
                uint32_t q_col = tmem + T_Q;
                uint64_t k_desc = next_slot(), q_desc = smem_desc(base + Q_AT, 16, 1024);
#pragma unroll 1
                for (int b = 0; b < Q_TMEM; ++b, k_desc += BLOCK >> 4, q_col += 32)
#pragma unroll
                    for (int x = 0; x < 4; ++x)      // 16 values a step: 32 bytes, 8 columns
                        pair_mma_ts(d, q_col + x * 8, k_desc + x * 2, qk, b + x > 0);
                if (!wait(sm.keys[slot], slot_phase)) break;
                k_desc = next_slot();
#pragma unroll 1
                for (int b = Q_TMEM; b < 9; ++b, k_desc += BLOCK >> 4, q_desc += BLOCK >> 4) {
                    if (b == 8) {
                        if (!wait(sm.rope, n & 1)) break;
                        k_desc = smem_desc(base + ROPE_AT, 16, 1024);
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) pair_mma(d, q_desc + x * 2, k_desc + x * 2, qk, true);
                }
                if (!ok) break;
                pair_commit(bar(sm.scored[n & 1]));
                begins = ++tile == w.tiles;
                if (begins) tile = 0;
            }
        } else {
            constexpr uint32_t pv = mma_desc(128, 256, DT == kBf16, true);
#pragma unroll 1
            for (int n = 0; ok && n < count; ++n) {
                wait(sm.values[n & 1], (n >> 1) & 1);
                if (!wait(sm.weighed, n & 1)) break;
                tc_fence_after();
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {            // 256 values a time
                    uint64_t p_desc = smem_desc(base + P_AT, 16, 1024), v_desc = smem_desc(base + slot * SLOT, BLOCK, 1024);
#pragma unroll 1
                    for (int y = 0; y < 2; ++y, p_desc += BLOCK >> 4, v_desc += PART >> 4)
#pragma unroll
                        for (int x = 0; x < 4; ++x)      // 16 keys a step
                            pair_mma(tmem + T_O + h * 128, p_desc + x * 2, v_desc + x * (2048 >> 4), pv, !begins || y + x > 0);
                    pair_commit(bar(sm.slot_free[slot]));
                    if (h == 1) pair_commit(bar(sm.added));
                    if (++slot == SLOTS) slot = 0;
                }
                begins = ++tile == w.tiles;
                if (begins) tile = 0;
            }
        }
        if (!ok) {     // let what was issued end before the pair goes
            const uint32_t drained = bar(sm.drained[warp - MMA_WARP]);
            pair_commit(drained);
            for (int i = 0; i < (1 << 20) && !mbar_try(drained, 0); ++i) {}
        }
    }
    __syncwarp();
    if (*gave_up) {      // let copies in flight come in (32 KB each, microseconds)
        uint64_t t0, t;
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
        do {
            asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
        } while (t - t0 < 1000000ull);
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive();      // no CTA leaves before the other has done with it
    cluster_wait();
    if (tid == 0 && sm.gave_up && a.status)
        for (int r = 0; r < a.R; ++r) record_status(a.status, r, kStatusAttendTimeout);
    if (warp == MMA_WARP) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ---- join ------------------------------------------------------------------------------

constexpr int JOIN_NT = 128;
constexpr int JOIN_WIDE = 1024;      // heads that get four warps each

// The parts of the heads of split groups, WARPS warps a head, a lane 16 / WARPS of its
// values; or, where there is no prefix (pairs 0), the heads' own parts alone.  Bound by
// latency: references and sums, and the values of the first parts, are loaded at once,
// and the values wait for nothing else.
template <int DT, int WARPS>
__global__ void __launch_bounds__(JOIN_NT, 4) join_kernel(const __grid_constant__ PrefixLaunch a, const __grid_constant__ PrefixParts w)
{
    constexpr int FOURS = 4 / WARPS, AT_ONCE = 16 / FOURS;      // of a lane's values; parts
    constexpr int LANES = (MAX_PAIRS + 31) / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = WARPS == 4 ? blockIdx.x : blockIdx.x * 4 + warp, four = WARPS == 4 ? threadIdx.x : lane;
    PrefixParts::Join join = {n / PAIR_HEADS, 0, 0};
    if (w.pairs > 0) join = w.join[n / PAIR_HEADS];
    const int head = join.group * PAIR_HEADS + n % PAIR_HEADS;
    const bool on = head < a.R * a.H;
    const int share = heads_of_cta(a.R * a.H, join.group);
    const int i = n % PAIR_HEADS < share ? n % PAIR_HEADS : n % PAIR_HEADS - share + CTA_HEADS;
    const HeadPlace at(a, on ? head : 0);
    // (a pair's second place is for the group that it has from its start)
    auto place = [&](int p) { return (int64_t)(join.first + p) * 2 + (p == 0); };
    auto values = [&](int p, int k) {
        return *reinterpret_cast<const float4 *>(w.o + place(p) * (PAIR_HEADS * kLatent * 4) + part_at(i, four + 32 * k));
    };
    uint8_t *out = a.out + at.r * a.out_rs + at.h * a.out_hs + four * 8;
    const uint8_t *own = a.part + at.r * a.part_rs + at.h * a.part_hs + four * 8;
    after_launch_before();
    if (!on) return;      // (all of the head's warps)
    float4 v[AT_ONCE][FOURS];
#pragma unroll
    for (int p = 0; p < AT_ONCE; ++p)
#pragma unroll
        for (int k = 0; k < FOURS; ++k)
            if (p < join.parts) v[p][k] = values(p, k);
    float2 ml[LANES];
    float m = -INFINITY, l = 0.0f, f[LANES], other = -INFINITY;
#pragma unroll
    for (int k = 0; k < LANES; ++k) {
        const int p = k * 32 + lane;
        ml[k] = p < join.parts ? w.ml[place(p) * PAIR_HEADS + i] : make_float2(-INFINITY, 0.0f);
    }
    uint2 part[FOURS];
    if (a.part) {
        other = a.part_lse[head];
#pragma unroll
        for (int k = 0; k < FOURS; ++k) part[k] = *reinterpret_cast<const uint2 *>(own + k * 256);
    }
#pragma unroll
    for (int k = 0; k < LANES; ++k) m = fmaxf(m, ml[k].x);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
#pragma unroll
    for (int k = 0; k < LANES; ++k) {
        f[k] = ex2(ml[k].x - (m == -INFINITY ? 0.0f : m));
        if (k * 32 + lane < join.parts) l = fmaf(f[k], ml[k].y, l);
    }
#pragma unroll
    for (int d = 1; d < 32; d *= 2) l += __shfl_xor_sync(0xffffffffu, l, d);
    float o[FOURS][4] = {};
#pragma unroll 1
    for (int p0 = 0; p0 < join.parts; p0 += AT_ONCE) {
        if (p0 > 0) {
#pragma unroll
            for (int p = 0; p < AT_ONCE; ++p)
#pragma unroll
                for (int k = 0; k < FOURS; ++k)
                    if (p0 + p < join.parts) v[p][k] = values(p0 + p, k);
        }
        // (AT_ONCE divides 32: the factors of a round are in one of f)
        const float fs = p0 < 32 ? f[0] : p0 < 64 ? f[1] : f[2];
#pragma unroll
        for (int p = 0; p < AT_ONCE; ++p) {
            const float by = __shfl_sync(0xffffffffu, fs, (p0 + p) & 31);
            if (p0 + p < join.parts) {
#pragma unroll
                for (int k = 0; k < FOURS; ++k) {
                    o[k][0] = fmaf(by, v[p][k].x, o[k][0]);
                    o[k][1] = fmaf(by, v[p][k].y, o[k][1]);
                    o[k][2] = fmaf(by, v[p][k].z, o[k][2]);
                    o[k][3] = fmaf(by, v[p][k].w, o[k][3]);
                }
            }
        }
    }
    float weight = 0.0f, scale = 1.0f;
    if (a.part) scale = add_part(m, l, other, &weight);
    const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
    scale *= inv;
    const float by = weight * inv;
    // (part may be out, whose values are this lane's own; part_lse lse)
    if (WARPS > 1)
        __syncthreads();
    else
        __syncwarp();
#pragma unroll
    for (int k = 0; k < FOURS; ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) o[k][j] *= scale;
        if (weight != 0.0f) {
            const float2 x = pair_to_float<DT>(part[k].x), y = pair_to_float<DT>(part[k].y);
            o[k][0] = fmaf(x.x, by, o[k][0]);
            o[k][1] = fmaf(x.y, by, o[k][1]);
            o[k][2] = fmaf(y.x, by, o[k][2]);
            o[k][3] = fmaf(y.y, by, o[k][3]);
        }
        *reinterpret_cast<uint2 *>(out + k * 256) = make_uint2(floats_to_pair<DT>(o[k][0], o[k][1]), floats_to_pair<DT>(o[k][2], o[k][3]));
    }
    if (four == 0 && a.lse) a.lse[head] = log2_sum(m, l) * kLn2;
}

// ---- host ------------------------------------------------------------------------------

// What a group of heads that a pair begins costs it beside its tiles (queries, O out; 10
// to 13 thousand cycles), and a tile (2,650), in eighths of a tile.  Measured with 0, 16,
// 29 and 40: 37 x 40 heads over 5,003 rows 34.9, 29.8, 30.0 and 29.7 us, 32 x 128 over
// 8,192 69.5, 66.2, 66.4 and 64.7, 256 x 16 over 40,000 232.5, 230.1, 229.4 and 226.8.
constexpr int GROUP_COST = 40, TILE_COST = 8;

// Cuts the tiles so that no pair costs more than `most` (but one tile a pair at
// least); whether MAX_PAIRS are enough.
bool cut(PrefixParts &w, int64_t most)
{
    int group = 0, tile = 0;
    for (w.pairs = 0; group < w.groups; ++w.pairs) {
        if (w.pairs == MAX_PAIRS) return false;
        w.start[w.pairs] = {group, tile};
        int64_t left = most;
        for (bool first = true; group < w.groups; first = false) {
            int64_t n = (left - GROUP_COST) / TILE_COST;
            if (n < 1) {
                if (!first) break;
                n = 1;
            }
            if (n < w.tiles - tile) {
                tile += (int)n;
                break;
            }
            left -= GROUP_COST + (int64_t)(w.tiles - tile) * TILE_COST;
            ++group;
            tile = 0;
        }
    }
    w.start[w.pairs] = {group, 0};
    w.joins = 0;
    for (int p = 1; p < w.pairs; ++p) {
        if (w.start[p].tile == 0) continue;
        if (w.joins > 0 && w.join[w.joins - 1].group == w.start[p].group)
            ++w.join[w.joins - 1].parts;
        else
            w.join[w.joins++] = {w.start[p].group, (int16_t)(p - 1), 2};
    }
    return true;
}

// Cuts the tiles evenly: nearly the least cost a pair for which there are enough pairs.
void cut_evenly(PrefixParts &w)
{
    const int64_t all = (int64_t)w.tiles * w.groups * TILE_COST;
    // every pair begins a group, and every group is begun
    int64_t most = (all + (int64_t)GROUP_COST * (w.groups > MAX_PAIRS ? w.groups : MAX_PAIRS)) / MAX_PAIRS;
    most = most > GROUP_COST + TILE_COST ? most : GROUP_COST + TILE_COST;
    while (!cut(w, most)) most += TILE_COST / 2 + most / 32;
}

PrefixParts lay_out(int32_t R, int32_t H, int32_t len, uint8_t *ws, int64_t *bytes)
{
    PrefixParts w;
    w.tiles = (len + KEYS - 1) / KEYS;
    w.groups = (int)(((int64_t)R * H + PAIR_HEADS - 1) / PAIR_HEADS);
    w.pairs = (int)((int64_t)w.tiles * w.groups < MAX_PAIRS ? (int64_t)w.tiles * w.groups : MAX_PAIRS);      // at most
    int64_t n = 16;      // never empty
    w.o = ws + n;
    n += (int64_t)w.pairs * 2 * PAIR_HEADS * kLatent * 4;
    w.ml = reinterpret_cast<float2 *>(ws + n);
    n += (int64_t)w.pairs * 2 * PAIR_HEADS * 8;
    w.there = ws + n;
    n += (int64_t)w.tiles * 32;
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
        auto beside = [&](auto kernel) {      // (see launch_expand)
            if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        };
        beside(expand_kernel<kBf16, kRow4, 2>), beside(expand_kernel<kBf16, kRow8, 2>), beside(expand_kernel<kBf16, kRow16, 2>);
        beside(expand_kernel<kF16, kRow4, 2>), beside(expand_kernel<kF16, kRow8, 2>), beside(expand_kernel<kF16, kRow16, 2>);
        if (e != cudaSuccess) return e;
        known[dev].store(true, std::memory_order_release);
    }
    return cudaSuccess;
}

// Many rows: as many CTAs as there is work for, and L1 as large as it gets, which holds
// what is on its way (256 x 16 heads over 40,000 rows of 16 bits: 226 us, 230 with the
// other kernel's).  Few: shared memory as prefix_kernel wants it, as an SM changes that
// only when it is idle; and one CTA an SM if most of its warps have two rounds then (32 x
// 16 heads, 8,192 rows: 22.3 us, 23.1 with a round a warp; 37 x 40 heads, 5,003 rows, 27.9
// and 27.4 the other way round).  (The kernel before, of 256 threads and 32 rows a CTA,
// beside which there was no place: 25.0 and 29.8.)
int expand_rounds(int tiles) { return tiles * (KEYS / EX_ROWS) <= 2 * 2 * MAX_PAIRS * (EX_NT / 32) ? 2 : 1; }      // at most

int expand_ctas(int tiles)
{
    constexpr int SMS = 2 * MAX_PAIRS;
    const int all = (tiles * (KEYS / EX_ROWS) + EX_NT / 32 - 1) / (EX_NT / 32);
    return expand_rounds(tiles) == 2 && all > SMS + SMS / 2 ? SMS : all;
}

template <int DT, int ROW>
cudaError_t launch_expand(const PrefixLaunch &a, const PrefixParts &w, cudaStream_t s)
{
    const dim3 ctas(expand_ctas(w.tiles));
    if (expand_rounds(w.tiles) == 2) return launch_behind(expand_kernel<DT, ROW, 2>, ctas, EX_NT, 0, 1, s, a, w);
    return launch_behind(expand_kernel<DT, ROW, 1>, ctas, EX_NT, 0, 1, s, a, w);
}

template <int DT>
cudaError_t launch(const PrefixLaunch &a, const PrefixParts &w, cudaStream_t s)
{
    if (w.pairs > 0) {
        cudaError_t e = a.row_bytes == kRow4 ? launch_expand<DT, kRow4>(a, w, s) : a.row_bytes == kRow8 ? launch_expand<DT, kRow8>(a, w, s) : launch_expand<DT, kRow16>(a, w, s);
        if (e != cudaSuccess) return e;
        e = launch_behind(prefix_kernel<DT>, dim3(w.pairs * 2), PX_NT, PX_SMEM, 2, s, a, w);
        if (e != cudaSuccess) return e;
        if (w.joins == 0) return e;
    }
    // Four warps a head where there are few, with many parts each (8,192 rows and 32 x 16
    // heads: 22.9 us, with one 23.4; 16 x 64: 29.5 and 31.5), else one (16 x 128: 39.6 us, with
    // four 42.3).
    const int heads = (w.pairs > 0 ? w.joins : w.groups) * PAIR_HEADS;
    if (heads <= JOIN_WIDE) return launch_behind(join_kernel<DT, 4>, dim3(heads), JOIN_NT, 0, 1, s, a, w);
    return launch_behind(join_kernel<DT, 1>, dim3(heads / 4), JOIN_NT, 0, 1, s, a, w);
}

}  // namespace

void attend_prefix_workspace_bytes(int32_t R, int32_t H, int32_t len, int64_t *bytes) { lay_out(R, H, len, nullptr, bytes); }

cudaError_t launch_attend_prefix(const PrefixLaunch &a, cudaStream_t s)
{
    const cudaError_t e = prepare_device();
    if (e != cudaSuccess) return e;
    int64_t bytes;
    PrefixParts w = lay_out(a.R, a.H, a.len, a.workspace, &bytes);
    if (w.pairs > 0) cut_evenly(w);
    return a.dtype == kBf16 ? launch<kBf16>(a, w, s) : launch<kF16>(a, w, s);
}

}  // namespace hs
