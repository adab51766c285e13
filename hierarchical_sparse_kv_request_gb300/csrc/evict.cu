// evict.cu -- eviction by accumulated attention weight: choose, per request,
// the hot slots whose tokens have gathered the least weight, and (with a
// handle's hot state) free them.
//
// One CTA per request.  A slot's key is its token's weight as a 32-bit
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
// Measured on GB300: 32 requests of 6,144 slots, 40,000 tokens 8.8 us, 256 of
// 32,768 slots 53 us.
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

struct EvictSmem {
    uint32_t hist[2048];
    uint32_t less[33 * 32], tied[33 * 32];   // bitmaps over slots (D <= 32 * EV_NT)
    uint32_t pos[EV_NT];                 // output place of each word's first chosen slot
    uint32_t zero[EV_NT];                // bitmap: stamp 0 after the call
    uint32_t warp_tot[EV_NT / 32];
    uint32_t bin, before, in_bin;
};

__device__ __forceinline__ uint32_t warp_inclusive_scan(uint32_t x, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// Finds the bin of the histogram in which the need-th key lies: sm.bin, with
// sm.before keys in the bins before it and sm.in_bin in it.  Returns the number
// of keys; need is brought down to it.  Clears the histogram.  Begins and ends
// with a barrier.
__device__ __forceinline__ uint32_t find_bin(EvictSmem &sm, uint32_t &need, int tid)
{
    const int lane = tid & 31, warp = tid >> 5;
    __syncthreads();
    uint2 &mine = reinterpret_cast<uint2 *>(sm.hist)[tid];
    const uint2 h = mine;
    const uint32_t sum = __reduce_add_sync(0xffffffffu, h.x + h.y);
    if (lane == 0) sm.warp_tot[warp] = sum;
    mine = make_uint2(0, 0);
    __syncthreads();
    const uint32_t upto = warp_inclusive_scan(sm.warp_tot[lane], lane);
    const uint32_t total = __shfl_sync(0xffffffffu, upto, 31);
    need = min(need, total);
    const uint32_t reached = __ballot_sync(0xffffffffu, upto >= need);
    if (need > 0 && __ffs(reached) - 1 == warp) {
        const uint32_t in = warp_inclusive_scan(h.x + h.y, lane) + __shfl_sync(0xffffffffu, upto, warp) - sum;
        if (__ffs(__ballot_sync(0xffffffffu, in >= need)) - 1 == lane) {
            const bool second = need > in - h.y;
            sm.bin = 2 * tid + second;
            sm.before = second ? in - h.y : in - h.y - h.x;
            sm.in_bin = second ? h.y : h.x;
        }
    }
    __syncthreads();
    return total;
}

// KT: slots per thread, D <= KT * EV_NT.  FREE: with a hot state.
template <int KT, bool FREE>
__global__ void __launch_bounds__(EV_NT) evict_kernel(EvictLaunch a)
{
    __shared__ EvictSmem sm;
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = a.D, n = a.n;
    const int32_t *s2t = a.slot2tok + (int64_t)r * D;
    const int32_t S = a.seq_lens[r];
    uint32_t key[KT];        // first its slot's token, then the token's weight
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        const int s = tid + i * EV_NT;
        key[i] = s < D ? (uint32_t)s2t[s] : kNoCandidate;
    }
    int32_t *out = a.out_slots ? a.out_slots + (int64_t)r * n : nullptr;
    uint32_t need = (uint32_t)max(0, a.want ? min(n, a.want[r]) : n);
    reinterpret_cast<uint2 *>(sm.hist)[tid] = make_uint2(0, 0);

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
        if (FREE && ok && a.protect_calls) ok = lu[tid + i * EV_NT] < thr;
        if (ok) candidates |= 1u << i;
    }
#pragma unroll
    for (int i = 0; i < KT; ++i)
        if (candidates >> i & 1u) key[i] = __float_as_uint(wt[key[i]]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        key[i] = candidates >> i & 1u ? weight_key(__uint_as_float(key[i])) : kNoCandidate;
        if (key[i] != kNoCandidate) atomicAdd(&sm.hist[key[i] >> 21], 1u);
    }
    find_bin(sm, need, tid);
    const int m = (int)need;
    if (m == 0) {     // the same for the whole CTA
        for (int i = tid; out && i < n; i += EV_NT) out[i] = -1;
        if (tid == 0 && a.out_counts) a.out_counts[r] = 0;
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
#pragma unroll
        for (int i = 0; i < KT; ++i)
            if (key[i] != kNoCandidate && (key[i] ^ T) >> digits_left == 0)
                atomicAdd(&sm.hist[key[i] >> shift & digits], 1u);
        find_bin(sm, need, tid);
        T |= sm.bin << shift;
        need -= sm.before;
        digits_left = shift;
    }
    const bool ties = sm.in_bin != need;
    if (!ties) T = min(T | ((1u << digits_left) - 1u), kNoCandidate - 1u);

    // bitmaps in slot order, and where each word's chosen slots go
    // (word i * 32 + warp is at warp * 33 + i: no bank conflicts either way)
    uint32_t less = 0, tied = 0;
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        const uint32_t b = __ballot_sync(0xffffffffu, ties ? key[i] < T : key[i] <= T);
        if (lane == i) less = b;
    }
    if (ties) {
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const uint32_t b = __ballot_sync(0xffffffffu, key[i] == T);
            if (lane == i) tied = b;
        }
    }
    sm.less[warp * 33 + lane] = less;
    sm.tied[warp * 33 + lane] = tied;
    __syncthreads();
    {
        less = sm.less[lane * 33 + warp];
        tied = sm.tied[lane * 33 + warp];
        const uint32_t l = __popc(less), t = __popc(tied);
        uint32_t tot;
        const uint32_t pre = block_exclusive_scan<EV_NT>((t << 16) | l, sm.warp_tot, tot);
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
            for (; chosen; chosen &= chosen - 1u) out[at++] = tid * 32 + __ffs(chosen) - 1;
            for (int i = m + tid; i < n; i += EV_NT) out[i] = -1;
        }
    }
    if (tid == 0 && a.out_counts) a.out_counts[r] = m;
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

template <int KT>
cudaError_t launch_kt(const EvictLaunch &a, cudaStream_t s)
{
    if (a.st.tok2slot)
        evict_kernel<KT, true><<<a.R, EV_NT, 0, s>>>(a);
    else
        evict_kernel<KT, false><<<a.R, EV_NT, 0, s>>>(a);
    return cudaGetLastError();
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
