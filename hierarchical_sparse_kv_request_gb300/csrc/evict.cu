// evict.cu -- eviction by accumulated attention weight: choose, per request,
// the hot slots whose tokens have gathered the least weight, and (with a
// handle's hot state) free them.
//
// One CTA per request.  A slot's key is its token's weight as a 32-bit
// integer of the same order (no candidate: the largest key), held in
// registers, slot s by thread s % NT.  The want-th smallest key T is found by
// a radix select (digits of 11, 11 and 10 bits, a shared-memory histogram
// each); the chosen slots are those with a key below T and the lowest slots
// among those equal to T, which is ascending (weight, slot) without a sort.
// Chosen and tied slots become two bitmaps in slot order (one ballot per 32
// slots), and one block scan over their words gives every chosen slot its
// place.
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
    uint32_t less[EV_NT], tied[EV_NT];   // bitmaps over slots (D <= 32 * EV_NT)
    uint32_t pos[EV_NT];                 // output place of each word's first chosen slot
    uint32_t zero[EV_NT];                // bitmap: stamp 0 after the call
    uint32_t warp_tot[EV_NT / 32];
    uint32_t bin, before;
};

// KT: slots per thread, D <= KT * EV_NT.  FREE: with a hot state.
template <int KT, bool FREE>
__global__ void __launch_bounds__(EV_NT) evict_kernel(EvictLaunch a)
{
    __shared__ EvictSmem sm;
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const int D = a.D, n = a.n;
    const int32_t S = a.seq_lens[r];
    int32_t *out = a.out_slots ? a.out_slots + (int64_t)r * n : nullptr;
    int want = n;
    if (a.want) want = max(0, min(n, a.want[r]));

    // keys
    const int32_t *s2t = a.slot2tok + (int64_t)r * D;
    const float *wt = a.weights + (int64_t)r * a.weights_stride;
    const int64_t horizon = S > D ? min((int64_t)S - a.keep_recent, a.weights_tokens) : 0;
    uint32_t thr = 0xFFFFFFFFu;
    if (FREE && a.protect_calls) {
        const uint32_t tick = a.st.tick[r];
        thr = tick >= a.protect_calls ? tick - a.protect_calls + 1u : 1u;
    }
    const uint32_t *lu = FREE ? a.st.last_used + (int64_t)r * D : nullptr;
    uint32_t key[KT];
    int32_t tok[KT];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        const int s = tid + i * EV_NT;
        tok[i] = s < D && horizon > 0 ? s2t[s] : -1;
    }
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        const int s = tid + i * EV_NT;
        key[i] = kNoCandidate;
        bool ok = tok[i] >= 0 && tok[i] < horizon;
        if (FREE && ok && a.protect_calls) ok = lu[s] < thr;
        if (ok) key[i] = weight_key(wt[tok[i]]);
        mine += ok;
    }
    uint32_t candidates;
    block_exclusive_scan<EV_NT>((uint32_t)mine, sm.warp_tot, candidates);
    const int m = min(want, (int)candidates);
    if (m <= 0) {     // the same for the whole CTA
        for (int i = tid; out && i < n; i += EV_NT) out[i] = -1;
        if (tid == 0 && a.out_counts) a.out_counts[r] = 0;
        return;
    }

    // T = the m-th smallest key; `need` of the keys equal to T are chosen
    uint32_t prefix = 0, mask = 0, need = (uint32_t)m;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digits = pass == 2 ? 1024u : 2048u;
        for (int b = tid; b < 2048; b += EV_NT) sm.hist[b] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < KT; ++i)
            if (key[i] != kNoCandidate && (key[i] & mask) == prefix)
                atomicAdd(&sm.hist[(key[i] >> shift) & (digits - 1u)], 1u);
        __syncthreads();
        const uint32_t h0 = sm.hist[2 * tid], h1 = sm.hist[2 * tid + 1];
        uint32_t tot;
        const uint32_t pre = block_exclusive_scan<EV_NT>(h0 + h1, sm.warp_tot, tot);
        if (pre < need && need <= pre + h0 + h1) {   // one thread
            const bool second = need > pre + h0;
            sm.bin = 2 * tid + second;
            sm.before = pre + (second ? h0 : 0u);
        }
        __syncthreads();
        need -= sm.before;
        prefix |= sm.bin << shift;
        mask |= (digits - 1u) << shift;
        __syncthreads();
    }
    const uint32_t T = prefix;

    // bitmaps in slot order, and where each word's chosen slots go
    if (tid < EV_NT) sm.less[tid] = sm.tied[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        const uint32_t l = __ballot_sync(0xffffffffu, key[i] < T);
        const uint32_t t = __ballot_sync(0xffffffffu, key[i] == T);
        if (lane == 0) {
            sm.less[i * 32 + (tid >> 5)] = l;
            sm.tied[i * 32 + (tid >> 5)] = t;
        }
    }
    __syncthreads();
    {
        const uint32_t l = __popc(sm.less[tid]), t = __popc(sm.tied[tid]);
        uint32_t tot;
        const uint32_t pre = block_exclusive_scan<EV_NT>((t << 16) | l, sm.warp_tot, tot);
        // of the ties, the lowest `need` slots are chosen
        const uint32_t tb = min(pre >> 16, need);
        sm.pos[tid] = (pre & 0xFFFFu) + tb;
        uint32_t bits = sm.tied[tid], left = need - tb, keep = 0;
        if (left >= t) {
            keep = bits;
        } else {
            for (; left; --left) {
                keep |= bits & (0u - bits);
                bits &= bits - 1u;
            }
        }
        sm.tied[tid] = sm.less[tid] | keep;       // now: the chosen slots
    }
    __syncthreads();
    const uint32_t below = (1u << lane) - 1u;
    if (out) {
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const int w = i * 32 + (tid >> 5);
            const uint32_t c = sm.tied[w];
            if ((c >> lane) & 1u) out[sm.pos[w] + __popc(c & below)] = tid + i * EV_NT;
        }
        for (int i = m + tid; i < n; i += EV_NT) out[i] = -1;
    }
    if (tid == 0 && a.out_counts) a.out_counts[r] = m;
    if (!FREE) return;

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
