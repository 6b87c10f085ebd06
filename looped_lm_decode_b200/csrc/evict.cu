// Eviction from a bf16 cache by accumulated attention weight.
//
// The library's own operator (the LoopVQ paper has no counterpart): a (sequence, KV head) whose length passes a
// budget keeps its sinks, its most recent tokens and, of the others, those with the highest scores (the weights
// that loopvq_bf16_decode_attn_scored accumulates).
//
// Keys are stored rotated, so attention does not depend on the slots' order, and a token may move to any slot:
// the i-th emptied slot below the budget takes the i-th kept token at or behind it.  Only the rows that change
// place move (one per head when one token is evicted, where an order-preserving compaction would move up to the
// whole cache), sources (slots >= budget) and targets (slots < budget) are disjoint, so every row moves in
// parallel and nothing is staged.
//
// Selection: scores map to unsigned keys in their own order (radix order of the fp32 bits, NaN lowest, protected
// tokens highest).  One CTA per (sequence, KV head) finds the budget-th largest key digit by digit from the top
// (11 + 11 + 10 bits, histograms in shared memory: integer counts, so the atomics' order does not matter), then
// every warp walks its own run of slots and ranks ties, emptied slots and moved tokens by ballots.
#include "loopvq_internal.cuh"

namespace loopvq {

namespace {

constexpr int kBins = 2048;

__device__ __forceinline__ uint32_t score_key(float s, int pos, int n_sink, long long recent_from) {
    if (pos < n_sink || pos >= recent_from) return 0xffffffffu;
    if (s != s) return 0u;
    const uint32_t u = __float_as_uint(s + 0.f);                     // -0 counts as +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of one value per warp, for every warp (NW <= 32); total in `sum`.  All threads call it.
template <int NW>
__device__ __forceinline__ int warps_prefix(int v, int *slots, int &sum) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) slots[warp] = v;
    __syncthreads();
    int before = 0;
    sum = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const int x = slots[w];
        before += w < warp ? x : 0;
        sum += x;
    }
    return before;
}

template <int NT, bool CACHED>
__global__ void __launch_bounds__(NT) evict_select_kernel(const EvictArgs a) {
    constexpr int NW = NT / 32;
    extern __shared__ uint32_t cached[];                             // CACHED: the keys of all slots
    __shared__ int hist[kBins];
    __shared__ int slots[NW];
    __shared__ int s_digit, s_above;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bh = blockIdx.x, b = bh / a.Hkv;
    const int len = min(max(__ldg(a.lens_in + b), 0), a.max_len);
    const size_t row = (size_t)bh * a.Nmax;
    const float *score = a.score_in + row;
    const int32_t *pos = a.pos_in + row;
    float *score_out = a.score_out + row;
    int32_t *pos_out = a.pos_out + row;
    if (len <= a.budget) {                                           // nothing to evict
        if (tid == 0) a.ws[bh] = 0;
        for (int n = tid; n < len; n += NT) {
            if (a.score_out != a.score_in) score_out[n] = score[n];
            if (a.pos_out != a.pos_in) pos_out[n] = pos[n];
        }
        return;
    }
    const long long recent_from = (long long)__ldg(a.next_pos + b) - a.n_recent;
    auto key_of = [&](int n) -> uint32_t {
        if constexpr (CACHED) return cached[n];
        return score_key(score[n], pos[n], a.n_sink, recent_from);
    };
    if constexpr (CACHED) {
        for (int n = tid; n < len; n += NT) cached[n] = score_key(score[n], pos[n], a.n_sink, recent_from);
    }

    // ---- the budget-th largest key: `prefix` under `mask`, of which `need` still have to be found
    uint32_t prefix = 0, mask = 0;
    int need = a.budget;
    const int shifts[3] = {21, 10, 0};
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = shifts[pass], bins = pass == 2 ? 1024 : 2048;
        __syncthreads();
        for (int i = tid; i < bins; i += NT) hist[i] = 0;
        __syncthreads();
        for (int n = tid; n < len; n += NT) {
            const uint32_t k = key_of(n);
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
        }
        __syncthreads();
        // the digit whose suffix count reaches `need`: every thread sums a run of bins, from the highest down
        const int per = bins / NT > 0 ? bins / NT : 1;
        int mine = 0;
        const int hi = bins - 1 - tid * per;                         // this thread's highest bin
        for (int i = 0; i < per; ++i)
            if (hi - i >= 0) mine += hist[hi - i];
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        int total;
        const int before = warps_prefix<NW>(__shfl_sync(0xffffffffu, inc, 31), slots, total);
        int above = before + inc - mine;                             // keys in higher bins
        if (above < need && above + mine >= need) {
            for (int i = 0; i < per; ++i) {
                const int c = hist[hi - i];
                if (above + c >= need) {
                    s_digit = hi - i;
                    s_above = above;
                    break;
                }
                above += c;
            }
        }
        __syncthreads();
        prefix |= (uint32_t)s_digit << shift;
        mask |= (uint32_t)(bins - 1) << shift;
        need -= s_above;
    }

    // ---- kept: keys above the threshold, and the `need` lowest slots among those equal to it
    const int run = ((len + NT - 1) / NT) * 32;                      // slots per warp, whole rounds
    const int w0 = min(warp * run, len), w1 = min(w0 + run, len);
    int ties = 0;
    for (int n0 = w0; n0 < w1; n0 += 32) {
        const int n = n0 + lane;
        ties += __popc(__ballot_sync(0xffffffffu, n < w1 && key_of(n) == prefix));
    }
    int unused;
    const int ties_before = warps_prefix<NW>(ties, slots, unused);
    const unsigned lower = (1u << lane) - 1u;
    int32_t *holes = a.ws + (size_t)a.B * a.Hkv + (size_t)bh * 2 * a.cap, *sources = holes + a.cap;
    int nh = 0, nsrc = 0, hole_base = 0, src_base = 0, moved = 0;
    for (int write = 0; write < 2; ++write) {
        int t = ties_before;
        nh = nsrc = 0;
        for (int n0 = w0; n0 < w1; n0 += 32) {
            const int n = n0 + lane;
            const bool in = n < w1;
            const uint32_t k = in ? key_of(n) : 0u;
            const unsigned eq = __ballot_sync(0xffffffffu, in && k == prefix);
            const bool kept = in && (k > prefix || (k == prefix && t + __popc(eq & lower) < need));
            t += __popc(eq);
            const bool hole = in && !kept && n < a.budget, source = kept && n >= a.budget;
            const unsigned mh = __ballot_sync(0xffffffffu, hole), ms = __ballot_sync(0xffffffffu, source);
            if (write) {
                if (hole) holes[hole_base + nh + __popc(mh & lower)] = n;
                if (source) sources[src_base + nsrc + __popc(ms & lower)] = n;
                if (kept && n < a.budget) {
                    if (a.score_out != a.score_in) score_out[n] = score[n];
                    if (a.pos_out != a.pos_in) pos_out[n] = pos[n];
                }
            }
            nh += __popc(mh);
            nsrc += __popc(ms);
        }
        if (!write) {
            hole_base = warps_prefix<NW>(nh, slots, moved);
            src_base = warps_prefix<NW>(nsrc, slots, unused);
        }
    }
    if (tid == 0) a.ws[bh] = moved;
}

// Rows of the moved tokens, their scores and positions; and the new lengths (the selection reads the old ones,
// which may be the same memory).  D / 8 lanes move a 16-byte piece each of a key row and a value row.
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;                                        // per CTA

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
    constexpr int NL = D / 8;
    constexpr int PER = kMoveThreads / NL;                           // rows in flight per CTA round
    const int bh = blockIdx.y, b = bh / a.Hkv;
    if (blockIdx.x == 0 && bh % a.Hkv == 0 && threadIdx.x == 0)
        a.lens_out[b] = min(min(max(a.lens_in[b], 0), a.max_len), a.budget);
    const int moved = a.ws[bh];
    const int32_t *holes = a.ws + (size_t)a.B * a.Hkv + (size_t)bh * 2 * a.cap, *sources = holes + a.cap;
    const size_t row = (size_t)bh * a.Nmax;
    const int lane = threadIdx.x % NL;
    const int end = min(moved, (int)(blockIdx.x + 1) * kMoveRows);
#pragma unroll 2
    for (int i = blockIdx.x * kMoveRows + threadIdx.x / NL; i < end; i += PER) {
        const size_t to = row + holes[i], from = row + sources[i];
        const uint4 kw = *reinterpret_cast<const uint4 *>(a.k + from * D + lane * 8);
        const uint4 vw = *reinterpret_cast<const uint4 *>(a.v + from * D + lane * 8);
        *reinterpret_cast<uint4 *>(a.k + to * D + lane * 8) = kw;
        *reinterpret_cast<uint4 *>(a.v + to * D + lane * 8) = vw;
        if (lane == 0) a.score_out[to] = a.score_in[from];
        if (lane == 1) a.pos_out[to] = a.pos_in[from];
    }
}

constexpr int kCachedKeys = 49152;                                   // 192 KiB of keys

template <int NT, bool CACHED>
cudaError_t launch_select(const EvictArgs &a, cudaStream_t s) {
    const size_t smem = CACHED ? (size_t)a.max_len * 4 : 0;
    auto kern = evict_select_kernel<NT, CACHED>;
    // the histogram's static shared memory counts against the same limit
    cudaError_t e = ensure_dynamic_smem((const void *)kern, smem + (kBins + 256) * sizeof(int));
    if (e != cudaSuccess) return e;
    kern<<<a.B * a.Hkv, NT, smem, s>>>(a);
    return cudaGetLastError();
}

int evict_cap(int max_len, int budget) {
    const int over = max_len > budget ? max_len - budget : 0;
    return over < budget ? over : budget;
}

}  // namespace

size_t evict_ws_bytes(int B, int Hkv, int max_len, int budget) {
    return (size_t)B * Hkv * (1 + 2 * (size_t)evict_cap(max_len, budget)) * sizeof(int32_t);
}

cudaError_t launch_evict(const EvictArgs &args, cudaStream_t s) {
    EvictArgs a = args;
    a.cap = evict_cap(a.max_len, a.budget);
    cudaError_t e = a.max_len > kCachedKeys ? launch_select<1024, false>(a, s)
                    : a.max_len > 4096      ? launch_select<1024, true>(a, s)
                                            : launch_select<256, true>(a, s);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((a.cap + kMoveRows - 1) / kMoveRows > 0 ? (a.cap + kMoveRows - 1) / kMoveRows : 1),
                    (unsigned)(a.B * a.Hkv));
    if (a.D == 128) evict_move_kernel<128><<<grid, kMoveThreads, 0, s>>>(a);
    else if (a.D == 64) evict_move_kernel<64><<<grid, kMoveThreads, 0, s>>>(a);
    else return cudaErrorInvalidValue;
    return cudaGetLastError();
}

}  // namespace loopvq
