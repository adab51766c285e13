// evict.cu -- eviction by accumulated attention weight: choose, per request,
// the hot slots whose tokens have gathered the least weight, and (with a
// handle's hot state) free them.
//
// One CTA per request, or a cluster of two (see as_pairs).  A slot's key is its token's weight as a 32-bit
// integer of the same order (no candidate: the largest key), held in
// registers, slot s by thread s % NT.  The want-th smallest key T is found by
// a radix select (digits of 11, 11 and 10 bits, a shared-memory histogram
// each, until a bin holds just the keys that are left to choose); the chosen
// slots are those with a key below T and the lowest slots among those equal to
// T, which is ascending (weight, slot) without a sort.  Chosen and tied slots
// become two bitmaps in slot order (one ballot per 32 slots), and one scan over
// their words gives every chosen slot its place.
//
// Bound by the gather of the weights by token, a 128-byte line of L1 a cycle
// and SM, and, below some 10,000 slots, by the latency of the steps.  Reading all
// of a request's weights into shared memory and gathering there was slower but
// for the largest buffers over the shortest contexts (256 requests, 81,920
// tokens: 16,384 slots 35 against 29.5 us, 32,768 slots 51 against 52.5).
// Measured on GB300: 32 requests of 6,144 slots, 40,000 tokens 8.2 us, 256 of
// 32,768 slots 52 us.
//
// Freeing keeps what the resolver relies on: the LRU list stays sorted by
// (last_used, slot).  A freed slot's stamp is 0, so the new list is all
// slots with stamp 0 in slot order, then the rest of the old list in its
// order ([Arch] "HiSparse local KV offload architecture", Hot lookup and LRU:
// victims come from the front).
#include "rows4.cuh"

namespace hs {
namespace {

constexpr int EV_NT = 1024;
constexpr uint32_t kNoCandidate = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w) return kNoCandidate - 1u;         // NaN: kept longest
    const uint32_t b = __float_as_uint(w + 0.0f); // -0 becomes 0
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// C: CTAs a request, a cluster of EV_NT threads between them.
template <int C>
struct EvictSmem {
    static constexpr int NT = EV_NT / C;
    uint32_t hist[C == 1 ? 1 : 3][2048];  // one a digit where the other CTA may still read it
    uint32_t less[33 * 32], tied[33 * 32];   // bitmaps over the CTA's slots (at most 32 * NT)
    uint32_t pos[C == 1 ? NT : 1];       // output place of each word's first chosen slot
    uint32_t zero[C == 1 ? NT : 1];      // bitmap: stamp 0 after the call
    uint32_t warp_tot[NT / 32];
    uint32_t bin, before, in_bin, chosen;
};

// What the cluster's CTAs have written before is there for each to read.
template <int C>
__device__ __forceinline__ void sync_ctas()
{
    if (C == 1) {
        __syncthreads();
    } else {
        __syncwarp();      // (.aligned: the warp together)
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
}

// The address in the cluster's other CTA (of two).
__device__ __forceinline__ uint32_t in_other(const void *p, int rank)
{
    uint32_t y;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(y) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank ^ 1));
    return y;
}

__device__ __forceinline__ uint32_t warp_inclusive_scan(uint32_t x, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// Finds the bin of the digit's histogram in which the need-th key lies: sm.bin,
// with sm.before keys in the bins before it and sm.in_bin in it, counting both
// CTAs' keys.  need is brought down to the number of keys.  Clears the
// histogram where it is used again.  Begins and ends with a barrier.
template <int C>
__device__ __forceinline__ void find_bin(EvictSmem<C> &sm, int digit, uint32_t &need, int tid, int rank)
{
    constexpr int BINS = 2 * C, WARPS = EvictSmem<C>::NT / 32;      // bins a thread
    const int lane = tid & 31, warp = tid >> 5;
    sync_ctas<C>();
    uint32_t *mine = sm.hist[C == 1 ? 0 : digit] + tid * BINS;
    uint32_t h[BINS];
    if (C == 1) {
        const uint2 x = *reinterpret_cast<uint2 *>(mine);
        h[0] = x.x, h[1] = x.y;
        *reinterpret_cast<uint2 *>(mine) = make_uint2(0, 0);
    } else {
        const uint4 x = *reinterpret_cast<uint4 *>(mine);
        uint4 y;
        asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w) : "r"(in_other(mine, rank)) : "memory");
        h[0] = x.x + y.x, h[1] = x.y + y.y, h[BINS - 2] = x.z + y.z, h[BINS - 1] = x.w + y.w;
    }
    uint32_t own = 0;
#pragma unroll
    for (int b = 0; b < BINS; ++b) own += h[b];
    const uint32_t sum = __reduce_add_sync(0xffffffffu, own);
    if (lane == 0) sm.warp_tot[warp] = sum;
    __syncthreads();
    const uint32_t upto = warp_inclusive_scan(lane < WARPS ? sm.warp_tot[lane] : 0u, lane);
    need = min(need, __shfl_sync(0xffffffffu, upto, 31));
    const uint32_t reached = __ballot_sync(0xffffffffu, upto >= need);
    if (need > 0 && __ffs(reached) - 1 == warp) {
        const uint32_t in = warp_inclusive_scan(own, lane) + __shfl_sync(0xffffffffu, upto, warp) - sum;
        if (__ffs(__ballot_sync(0xffffffffu, in >= need)) - 1 == lane) {
            uint32_t before = in - own;
            int b = 0;
#pragma unroll
            for (int u = 0; u < BINS - 1; ++u)
                if (b == u && before + h[u] < need) before += h[u], b = u + 1;
            sm.bin = BINS * tid + b;
            sm.before = before;
            uint32_t in_bin = h[0];
#pragma unroll
            for (int u = 1; u < BINS; ++u)
                if (b == u) in_bin = h[u];
            sm.in_bin = in_bin;
        }
    }
    __syncthreads();
}

// KT: slots per thread, D <= KT * EV_NT; a CTA has KT * NT neighbouring slots.
// FREE: with a hot state (one CTA).
template <int KT, bool FREE, int C>
__global__ void __launch_bounds__(EV_NT / C) evict_kernel(EvictLaunch a)
{
    static_assert(C == 1 || !FREE, "");
    constexpr int NT = EV_NT / C, WARPS = NT / 32;
    __shared__ __align__(16) EvictSmem<C> sm;
    const int r = C == 1 ? blockIdx.x : blockIdx.x / C, rank = C == 1 ? 0 : blockIdx.x % C;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = a.D, n = a.n, s0 = rank * KT * NT + tid;      // the thread's first slot
    const int32_t *s2t = a.slot2tok + (int64_t)r * D;
    after_launch_before();
    const int32_t S = a.seq_lens[r];
    uint32_t key[KT];        // first its slot's token, then the token's weight
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        const int s = s0 + i * NT;
        key[i] = s < D ? (uint32_t)s2t[s] : kNoCandidate;
    }
    int32_t *out = a.out_slots ? a.out_slots + (int64_t)r * n : nullptr;
    uint32_t need = (uint32_t)max(0, a.want ? min(n, a.want[r]) : n);
    for (int i = tid; i < (int)(sizeof(sm.hist) / 16); i += NT) reinterpret_cast<uint4 *>(sm.hist)[i] = make_uint4(0, 0, 0, 0);

    const float *wt = a.weights + (int64_t)r * a.weights_stride;
    const int32_t horizon = S > D ? (int32_t)max(min((int64_t)S - a.keep_recent, a.weights_tokens), (int64_t)0) : 0;
    uint32_t thr = 0xFFFFFFFFu;
    if (FREE && a.protect_calls) {
        const uint32_t tick = a.st.tick[r];
        thr = tick >= a.protect_calls ? tick - a.protect_calls + 1u : 1u;
    }
    const uint32_t *lu = FREE ? a.st.last_used + (int64_t)r * D : nullptr;
    uint32_t candidates = 0;     // bit i: slot i is one
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        bool ok = key[i] < (uint32_t)horizon;
        if (FREE && ok && a.protect_calls) ok = lu[s0 + i * NT] < thr;
        if (ok) candidates |= 1u << i;
    }
#pragma unroll
    for (int i = 0; i < KT; ++i)
        if (candidates >> i & 1u) key[i] = __float_as_uint(wt[key[i]]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        key[i] = candidates >> i & 1u ? weight_key(__uint_as_float(key[i])) : kNoCandidate;
        if (key[i] != kNoCandidate) atomicAdd(&sm.hist[0][key[i] >> 21], 1u);
    }
    find_bin<C>(sm, 0, need, tid, rank);
    const int m = (int)need;
    if (m == 0) {     // the same for the whole cluster
        for (int i = tid; rank == 0 && out && i < n; i += NT) out[i] = -1;
        if (tid == 0 && rank == 0 && a.out_counts) a.out_counts[r] = 0;
        if (C > 1) sync_ctas<C>();      // (its histogram has been read)
        return;
    }

    // Of the keys whose digits so far are T's, `need` are still to be chosen;
    // if that is all of them, the keys up to T (its other digits all ones) are.
    uint32_t T = sm.bin << 21;
    need -= sm.before;
    int digits_left = 21;
#pragma unroll 1
    while (sm.in_bin != need && digits_left > 0) {
        const int shift = digits_left == 21 ? 10 : 0;
        const uint32_t digits = (1u << (digits_left - shift)) - 1u;
        const int digit = C == 1 ? 0 : shift ? 1 : 2;
#pragma unroll
        for (int i = 0; i < KT; ++i)
            if (key[i] != kNoCandidate && (key[i] ^ T) >> digits_left == 0)
                atomicAdd(&sm.hist[digit][key[i] >> shift & digits], 1u);
        find_bin<C>(sm, digit, need, tid, rank);
        T |= sm.bin << shift;
        need -= sm.before;
        digits_left = shift;
    }
    const bool ties = sm.in_bin != need;
    // (no key is 0: that of -inf is 0x007FFFFF)
    const uint32_t upto = ties ? T - 1u : min(T | ((1u << digits_left) - 1u), kNoCandidate - 1u);

    // bitmaps in slot order, and where each word's chosen slots go
    // (word i * WARPS + warp is at warp * 33 + i: few bank conflicts either way)
    uint32_t less = 0, tied = 0;
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        const uint32_t b = __ballot_sync(0xffffffffu, key[i] <= upto);
        less = lane == i ? b : less;
    }
    if (ties) {
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const uint32_t b = __ballot_sync(0xffffffffu, key[i] == T);
            tied = lane == i ? b : tied;
        }
    }
    sm.less[warp * 33 + lane] = less;
    sm.tied[warp * 33 + lane] = tied;
    __syncthreads();
    {
        const int word = tid % WARPS * 33 + tid / WARPS;
        less = sm.less[word];
        tied = sm.tied[word];
        const uint32_t l = __popc(less), t = __popc(tied);
        uint32_t tot;
        uint32_t pre = block_exclusive_scan<NT>((t << 16) | l, sm.warp_tot, tot);
        if (C > 1) {      // behind the slots of the CTA before
            if (tid == 0) sm.chosen = tot;
            sync_ctas<C>();
            uint32_t other;
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(other) : "r"(in_other(&sm.chosen, rank)) : "memory");
            if (rank) pre += other;
        }
        // of the ties, the lowest `need` slots are chosen
        const uint32_t tb = min(pre >> 16, need);
        uint32_t left = need - tb, keep = 0;
        if (left >= t) {
            keep = tied;
        } else {
            for (; left; --left) {
                keep |= tied & (0u - tied);
                tied &= tied - 1u;
            }
        }
        uint32_t chosen = less | keep, at = (pre & 0xFFFFu) + tb;
        if (FREE) sm.tied[tid] = chosen;
        if (out) {
            for (; chosen; chosen &= chosen - 1u) out[at++] = rank * KT * NT + tid * 32 + __ffs(chosen) - 1;
            for (int i = m + tid + rank * NT; i < n; i += EV_NT) out[i] = -1;
        }
    }
    if (tid == 0 && rank == 0 && a.out_counts) a.out_counts[r] = m;
    if (C > 1) sync_ctas<C>();      // (its count has been read)
    if (!FREE) return;
    __syncthreads();
    const uint32_t below = (1u << lane) - 1u;

    // free the chosen slots; zero: the slots whose stamp is 0 afterwards
    int32_t *t2s = a.st.tok2slot + a.host_off[r];
    uint32_t *lu_w = a.st.last_used + (int64_t)r * D;
    uint32_t *res = a.st.resbits ? a.st.resbits + (int64_t)r * a.st.res_words : nullptr;
    uint16_t *lru = a.st.lru + (int64_t)r * D;
    for (int i = 0; i < KT; ++i) {
        const int s = tid + i * EV_NT, w = i * 32 + (tid >> 5);
        const bool freed = (sm.tied[w] >> lane) & 1u;
        const bool zero = freed || (s < D && lu_w[s] == 0u);
        if (freed) {
            int32_t *at = a.st.slot2tok + (int64_t)r * D + s;
            const int32_t t = *at;
            *at = -1;
            t2s[t] = -1;
            lu_w[s] = 0u;
            if (res) atomicAnd(&res[t >> 5], ~(1u << (t & 31)));
        }
        const uint32_t z = __ballot_sync(0xffffffffu, zero);
        if (lane == 0) sm.zero[w] = z;
    }
    __syncthreads();
    // the list entries that keep a stamp go behind the zeros, in their order
    auto stays = [&](int e, uint32_t &slot) {
        slot = e < D ? lru[e] : 0u;
        return e < D && !((sm.zero[slot >> 5] >> (slot & 31)) & 1u);
    };
    for (int i = 0; i < KT; ++i) {
        uint32_t slot;
        const uint32_t b = __ballot_sync(0xffffffffu, stays(tid + i * EV_NT, slot));
        if (lane == 0) sm.less[i * 32 + (tid >> 5)] = b;
    }
    __syncthreads();
    const uint32_t z = tid < KT * 32 ? sm.zero[tid] : 0u;
    const uint32_t s = tid < KT * 32 ? sm.less[tid] : 0u;
    uint32_t tot;
    const uint32_t pre = block_exclusive_scan<EV_NT>((__popc(z) << 16) | __popc(s), sm.warp_tot, tot);
    sm.pos[tid] = (tot >> 16) + (pre & 0xFFFFu);
    // An entry never moves forward in the list (the zeros only gain slots), so
    // from the back, with every thread's entry read before any is written,
    // none is overwritten before it is read.
    for (int i = KT - 1; i >= 0; --i) {
        uint32_t slot;
        const bool stay = stays(tid + i * EV_NT, slot);
        __syncthreads();
        const int w = i * 32 + (tid >> 5);
        if (stay) lru[sm.pos[w] + __popc(sm.less[w] & below)] = (uint16_t)slot;
    }
    __syncthreads();
    uint32_t at = pre >> 16;
    for (uint32_t bits = z; bits; bits &= bits - 1u) lru[at++] = (uint16_t)(tid * 32 + __ffs(bits) - 1);
}

// Whether the device has two SMs a request.  A request of more than 8,192 slots
// is then shared by two CTAs, each of which gathers half: measured for 32
// requests of 16,384 slots 10.9 against 13.9 us, of 32,768 slots 16.4 against
// 25.5.  Where CTAs have to share SMs it is slower (100 requests of 32,768 slots
// 28 against 26.5 us), and for fewer slots too (32 requests of 6,144 slots 7.9
// against 7.7).
cudaError_t as_pairs(int R, bool *yes)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    *yes = 2 * R <= sms;
    return e;
}

template <int KT>
cudaError_t launch_kt(const EvictLaunch &a, cudaStream_t s)
{
    if (a.st.tok2slot) return launch_behind(evict_kernel<KT, true, 1>, dim3(a.R), EV_NT, 0, 1, s, a);
    if (KT >= 16) {
        bool pairs;
        const cudaError_t e = as_pairs(a.R, &pairs);
        if (e != cudaSuccess) return e;
        if (pairs) return launch_behind(evict_kernel<KT < 16 ? 16 : KT, false, 2>, dim3(a.R * 2), EV_NT / 2, 0, 2, s, a);
    }
    return launch_behind(evict_kernel<KT, false, 1>, dim3(a.R), EV_NT, 0, 1, s, a);
}

}  // namespace

cudaError_t launch_evict(const EvictLaunch &a, cudaStream_t s)
{
    const int per = (a.D + EV_NT - 1) / EV_NT;
    if (per <= 1) return launch_kt<1>(a, s);
    if (per <= 2) return launch_kt<2>(a, s);
    if (per <= 4) return launch_kt<4>(a, s);
    if (per <= 8) return launch_kt<8>(a, s);
    if (per <= 16) return launch_kt<16>(a, s);
    return launch_kt<32>(a, s);
}

}  // namespace hs
