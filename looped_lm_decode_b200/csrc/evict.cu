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
// tokens highest), a key and its slot to one 64-bit rank (ties: the lower slot first), and one CTA per (sequence, KV
// head), or a cluster, finds the budget-th largest rank: a histogram of the keys' top 11 bits names the bin that holds
// it, and the few keys of that bin are ranked against one another; only if they are many (equal scores) do further
// digits follow, and then the slots' order.  Histograms are integer counts in shared memory and ranks are distinct, so
// the atomics' order does not matter.  Keys are read once and stay in registers; a long row is shared out over a cluster
// of up to 8 CTAs, which send one another their counts and lists.
//
// What bounds it: a step's eviction (32 sequences x 16 heads, 2049 slots to 2048: 9.0 us, 17 MB read and written) is a
// chain of latencies, 12000 clocks: loads 3500, histogram 1000, digit 1000, list 2500, marks 2800 (clocks that
// several CTAs of an SM share).  A long one (2 x 16 heads, 32768 slots to 4096: 41 us) selects in 20 us, of which the
// cluster's slowest loads are half (its CTAs wait for one another), and reads and writes 117 MB of rows of 256 bytes in 20.
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

// The slots' keys in the registers of their threads: warp w holds slots [w * ITEMS * 32, ...), lane-contiguous.  load()
// reads every slot that could be there before it knows how many are (their latency is the length's), and copies the slots
// that stay where the outputs are other memory.
template <int NT, int ITEMS>
struct RegKeys {
    uint32_t k[ITEMS];
    int base;
    __device__ __forceinline__ int load(const EvictArgs &a, size_t row, int b, int part, int) {
        constexpr int B = 5;                                         // pairs of loads in flight
        base = part * (NT * ITEMS) + (threadIdx.x >> 5) * (ITEMS * 32) + (threadIdx.x & 31);
        int len = word(a.lens_in + b);
        const long long from = (long long)word(a.next_pos + b) - a.n_recent;
        len = min(max(len, 0), a.max_len);
        const int stay = min(len, a.budget);
#pragma unroll
        for (int i0 = 0; i0 < ITEMS; i0 += B) {
            float s[B];
            int p[B];
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const int n = base + (i0 + i) * 32;
                s[i] = n < a.max_len ? a.score_in[row + n] : 0.f;
                p[i] = n < a.max_len ? a.pos_in[row + n] : 0;
            }
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const int n = base + (i0 + i) * 32;
                if (n < stay && a.score_out != a.score_in) a.score_out[row + n] = s[i];
                if (n < stay && a.pos_out != a.pos_in) a.pos_out[row + n] = p[i];
                k[i0 + i] = score_key(s[i], p[i], a.n_sink, from);
            }
        }
        return len;
    }
    template <typename F>
    __device__ __forceinline__ void each(int len, F f) const {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) f(base + i * 32, k[i], base + i * 32 < len);
    }
    // g(first slot, mask) for every 32 slots with the mask of those for which f holds; mark() replaces the keys by the
    // masks, marked() walks them again
    template <typename F, typename G>
    __device__ __forceinline__ void mark(int len, F f, G g) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int n = base + i * 32;
            k[i] = __ballot_sync(0xffffffffu, n < len && f(n, k[i]));
            g(n, k[i]);
        }
    }
    template <typename F, typename G>
    __device__ __forceinline__ void marked(int, F, G g) const {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) g(base + i * 32, k[i]);
    }
};

// Words sent to the same place of another CTA's shared memory in the cluster: sent, not fetched, so that nothing waits
// for a round trip (fetching the other CTAs' histograms took 17 us a row).
__device__ __forceinline__ uint32_t at_cta(const void *p, int rank) {
    uint32_t addr;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return addr;
}
__device__ __forceinline__ void to_cta(void *p, int rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at_cta(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void add_at_cta(void *p, int rank, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(at_cta(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync() {                     // (not .aligned: some calls come behind divergent loops)
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
template <int CL>
__device__ __forceinline__ void sync_row() {                         // the CTAs of a row
    if constexpr (CL > 1) cluster_sync();
    else __syncthreads();
}

// Any number of slots: keys computed again from memory (L2) at every use.
template <int NT>
struct MemKeys {
    const float *score;
    const int32_t *pos;
    int n_sink, base, count;
    long long from;
    __device__ __forceinline__ int load(const EvictArgs &a, size_t row, int b, int part, int parts) {
        const int len = min(max(word(a.lens_in + b), 0), a.max_len), stay = min(len, a.budget);
        score = a.score_in + row;
        pos = a.pos_in + row;
        n_sink = a.n_sink;
        from = (long long)word(a.next_pos + b) - a.n_recent;
        count = (len + NT * parts - 1) / (NT * parts);
        base = (part * (NT / 32) + (threadIdx.x >> 5)) * (count * 32) + (threadIdx.x & 31);
        const int end = min(stay, (part + 1) * count * NT);
        if (a.score_out != a.score_in)
            for (int n = part * count * NT + threadIdx.x; n < end; n += NT) a.score_out[row + n] = score[n];
        if (a.pos_out != a.pos_in)
            for (int n = part * count * NT + threadIdx.x; n < end; n += NT) a.pos_out[row + n] = pos[n];
        return len;
    }
    template <typename F>
    __device__ __forceinline__ void each(int len, F f) const {
        for (int i = 0; i < count; ++i) {
            const int n = base + i * 32;
            f(n, n < len ? score_key(score[n], pos[n], n_sink, from) : 0u, n < len);
        }
    }
    template <typename F, typename G>
    __device__ __forceinline__ void mark(int len, F f, G g) const {
        each(len, [&](int n, uint32_t k, bool in) { g(n, __ballot_sync(0xffffffffu, in && f(n, k))); });
    }
    template <typename F, typename G>
    __device__ __forceinline__ void marked(int len, F f, G g) const {
        mark(len, f, g);
    }
};

constexpr int kList = 512;                                           // keys of a bin that are ranked directly

// FUSED: few rows move, and this CTA moves them itself; the lengths are written here (behind a barrier of the cluster that
// holds a sequence's heads where they are written in place), so one launch does it all.
// CL: CTAs per row (a cluster where more than 1).
template <int NT, typename Keys, int FUSED_D, int CL>
__global__ void __launch_bounds__(NT, NT == 256 ? 4 : 2) evict_select_kernel(const EvictArgs a) {
    constexpr int NW = NT / 32;
    constexpr bool FUSED = FUSED_D > 0;
    static_assert(CL == 1 || !FUSED, "clusters of a row, or of a sequence's heads");
    static_assert(1024 % NT == 0, "runs of bins");
    __shared__ __align__(16) int hist[kBins];
    __shared__ int slots[NW];
    __shared__ int s_digit, s_above, s_count;
    __shared__ uint32_t s_rank[2];                                   // slot (complemented) and key of the bound
    __shared__ int s_each[3][CL];                                    // every CTA's list, emptied slots, moved tokens
    __shared__ __align__(16) int hist_all[CL > 1 ? kBins : 4];       // the cluster's histogram
    int *const bins_all = CL > 1 ? hist_all : hist;
    __shared__ uint4 list4[kList / 4];                               // a bin's keys in slot order; later the rows that move
    __shared__ int list_slot[kList];
    uint32_t *list = reinterpret_cast<uint32_t *>(list4);
    const int tid = threadIdx.x, lane = tid & 31;
    const int bh = blockIdx.x / CL, b = bh / a.Hkv;
    const int part = CL > 1 ? blockIdx.x % CL : 0;
    grid_trigger();
    grid_wait();
    const size_t row = (size_t)bh * a.Nmax;
    Keys keys;
    const int len = keys.load(a, row, b, part, CL);                            // and copies the slots that stay; emptied ones are
                                                                     // written again when their new tokens move in
    auto write_len = [&]() {
        if constexpr (FUSED) {
            if (a.lens_out == a.lens_in) {                           // every head of the sequence has read it
                cluster_sync();
            }
            if (tid == 0 && bh % a.Hkv == 0) a.lens_out[b] = min(len, a.budget);
        }
    };
    if (len <= a.budget) {                                           // nothing to evict
        if (!FUSED && tid == 0 && part == 0) a.ws[bh] = 0;
        write_len();
        return;
    }
    // ---- the budget-th largest rank: a prefix of the key under `mask`, of whose bin `need` are kept
    uint32_t prefix = 0, mask = 0;
    int need = a.budget;
    unsigned long long bound = 0;                                    // kept: rank >= bound
    const int shifts[3] = {21, 10, 0};
    bool found = false;
    for (int pass = 0; pass < 3 && !found; ++pass) {
        const int shift = shifts[pass], bins = pass == 2 ? 1024 : 2048;
        __syncthreads();
        for (int i = tid; i < bins / 4; i += NT) {
            reinterpret_cast<int4 *>(hist)[i] = make_int4(0, 0, 0, 0);
            if constexpr (CL > 1) reinterpret_cast<int4 *>(hist_all)[i] = make_int4(0, 0, 0, 0);
        }
        sync_row<CL>();
        keys.each(len, [&](int, uint32_t k, bool in) {
            if (in && (k & mask) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
        });
        __syncthreads();
        if constexpr (CL > 1) {                                      // few bins hold keys
            for (int i = tid; i < bins; i += NT) {
                const int c = hist[i];
                if (c > 0) {
#pragma unroll
                    for (int r = 0; r < CL; ++r) add_at_cta(&hist_all[i], r, (uint32_t)c);
                }
            }
            cluster_sync();
        }
        // the digit whose suffix count reaches `need`: every thread sums a run of bins, from the highest down
        const int per = bins / NT;
        int mine = 0;
        const int hi = bins - 1 - tid * per;                         // this thread's highest bin
        if (per % 4 == 0) {                                          // wide: single words of runs meet in few banks
            const int4 *run = reinterpret_cast<const int4 *>(bins_all + hi + 1 - per);
            for (int i = 0; i < per / 4; ++i) {
                const int4 c = run[i];
                mine += c.x + c.y + c.z + c.w;
            }
        } else {
            for (int i = 0; i < per; ++i) mine += bins_all[hi - i];
        }
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
                const int c = bins_all[hi - i];
                if (above + c >= need) {
                    s_digit = hi - i;
                    s_above = above;
                    s_count = c;
                    break;
                }
                above += c;
            }
        }
        __syncthreads();
        prefix |= (uint32_t)s_digit << shift;
        mask |= (uint32_t)(bins - 1) << shift;
        need -= s_above;
        const int count = s_count;
        if (count == need) {                                         // the whole bin is kept
            bound = (unsigned long long)prefix << 32;
            found = true;
        } else if (count <= kList) {
            int first = 0, last;                                     // this CTA's keys in the list
            auto found_at = [&](int i) {
                const uint32_t slot = ~(uint32_t)list_slot[i], k = list[i];
#pragma unroll
                for (int r = 0; r < CL; ++r) {
                    if constexpr (CL > 1) {
                        to_cta(&s_rank[0], r, slot);
                        to_cta(&s_rank[1], r, k);
                    } else {
                        s_rank[0] = slot;
                        s_rank[1] = k;
                    }
                }
            };
            // places by counting (one shared counter would take the keys one by one)
            int mine2 = 0, own;
            keys.each(len, [&](int, uint32_t k, bool in) {
                mine2 += __popc(__ballot_sync(0xffffffffu, in && (k & mask) == prefix));
            });
            int at = warps_prefix<NW>(mine2, slots, own);
            if constexpr (CL > 1) {                                  // behind the lists of the CTAs before
                if (tid < CL) to_cta(&s_each[0][part], tid, (uint32_t)own);
                cluster_sync();
                for (int r = 0; r < part; ++r) first += s_each[0][r];
                at += first;
                last = first + own;
            } else {
                last = count;
            }
            if (mine2 > 0) {
                keys.each(len, [&](int n, uint32_t k, bool in) {
                    const bool hit = in && (k & mask) == prefix;
                    const unsigned m = __ballot_sync(0xffffffffu, hit);
                    if (hit) {
                        const int i = at + __popc(m & ((1u << lane) - 1u));
                        if constexpr (CL > 1) {
#pragma unroll
                            for (int r = 0; r < CL; ++r) to_cta(&list[i], r, k);
                        } else {
                            list[i] = k;
                        }
                        list_slot[i] = n;                            // ranked where it is
                    }
                    at += __popc(m);
                });
            }
            if (tid < 3 && count + tid < kList) list[count + tid] = 0;
            sync_row<CL>();
            if (__syncthreads_and(tid >= count || (list[tid % kList] == list[0] && (count <= NT || list[(tid + NT) % count] == list[0])))) {
                if (tid == 0 && need - 1 >= first && need - 1 < last) found_at(need - 1);   // all equal (scores of 0, say)
            } else {
                // a key's place: larger ones and, before it, equal ones.  `parts` neighbouring threads share its comparisons
                const int own2 = last - first;
                int parts = 1;
                while (parts < 32 && own2 * parts * 2 <= NT) parts *= 2;
                const int quads = (count + 3) / 4;
                for (int i0 = first; i0 < last; i0 += NT / parts) {
                    const bool live = i0 + tid / parts < last;
                    const int i = live ? i0 + tid / parts : first, share = tid % parts;   // (behind the list: not read)
                    const uint32_t mine = list[i];
                    int higher = 0, j = share;
#pragma unroll 4
                    for (; j < i / 4 && j < quads; j += parts) {     // earlier slots
                        const uint4 y = list4[j];
                        higher += (y.x >= mine) + (y.y >= mine) + (y.z >= mine) + (y.w >= mine);
                    }
                    if (j == i / 4) {
                        const uint4 y = list4[j];
                        higher += (i % 4 > 0 ? y.x >= mine : y.x > mine) + (i % 4 > 1 ? y.y >= mine : y.y > mine) +
                                  (i % 4 > 2 ? y.z >= mine : y.z > mine) + (y.w > mine);
                        j += parts;
                    }
#pragma unroll 4
                    for (; j < quads; j += parts) {                  // later ones; behind the last: zeros
                        const uint4 y = list4[j];
                        higher += (y.x > mine) + (y.y > mine) + (y.z > mine) + (y.w > mine);
                    }
                    for (int o = 1; o < parts; o <<= 1) higher += __shfl_xor_sync(0xffffffffu, higher, o);
                    if (live && share == 0 && higher == need - 1) found_at(i);
                }
            }
            sync_row<CL>();
            bound = ((unsigned long long)s_rank[1] << 32) | s_rank[0];
            found = true;
        }
    }
    if (!found) {
        // many equal keys: the `need` lowest slots of them, counted in the slots' order
        int ties = 0;
        keys.each(len, [&](int, uint32_t k, bool in) { ties += __popc(__ballot_sync(0xffffffffu, in && k == prefix)); });
        int all;
        int t = warps_prefix<NW>(ties, slots, all);
        if constexpr (CL > 1) {
            if (tid < CL) to_cta(&s_each[0][part], tid, (uint32_t)all);
            cluster_sync();
            for (int r = 0; r < part; ++r) t += s_each[0][r];
        }
        keys.each(len, [&](int n, uint32_t k, bool in) {
            const unsigned eq = __ballot_sync(0xffffffffu, in && k == prefix);
            if (in && k == prefix && t + __popc(eq & ((1u << lane) - 1u)) == need - 1) {
                if constexpr (CL > 1) {
                    for (int r = 0; r < CL; ++r) {
                        to_cta(&s_rank[0], r, ~(uint32_t)n);
                        to_cta(&s_rank[1], r, k);
                    }
                } else {
                    s_rank[0] = ~(uint32_t)n;
                    s_rank[1] = k;
                }
            }
            t += __popc(eq);
        });
        sync_row<CL>();
        bound = ((unsigned long long)s_rank[1] << 32) | s_rank[0];
    }

    // ---- emptied slots below the budget and moved tokens behind it, both in ascending order
    const unsigned lower = (1u << lane) - 1u;
    const uint32_t bound_key = (uint32_t)(bound >> 32), bound_slot = ~(uint32_t)bound;
    // a slot below the budget that is emptied, or one behind it that is kept
    auto changes = [&](int n, uint32_t k) {
        return (k > bound_key || (k == bound_key && (uint32_t)n <= bound_slot)) == (n >= a.budget);
    };
    auto below = [&](int n) {                                        // lanes whose slots lie below the budget
        const int c = a.budget - (n - lane);
        return c >= 32 ? 0xffffffffu : c <= 0 ? 0u : (1u << c) - 1u;
    };
    int32_t *holes = FUSED ? reinterpret_cast<int32_t *>(list4)
                           : a.ws + (size_t)a.B * a.Hkv + (size_t)bh * 2 * a.cap;
    int32_t *sources = holes + a.cap;
    if (FUSED) __syncthreads();                                      // the list has been read
    int nh = 0, nsrc = 0, moved, unused;
    keys.mark(len, changes, [&](int n, uint32_t m) {
        const uint32_t bm = below(n);
        nh += __popc(m & bm);
        nsrc += __popc(m & ~bm);
    });
    int hole_at = warps_prefix<NW>(nh, slots, moved);
    int src_at = warps_prefix<NW>(nsrc, slots, unused);
    if constexpr (CL > 1) {
        if (tid < CL) {
            to_cta(&s_each[1][part], tid, (uint32_t)moved);
            to_cta(&s_each[2][part], tid, (uint32_t)unused);
        }
        cluster_sync();                                              // the last: no CTA writes into another behind it
        moved = 0;
        for (int r = 0; r < CL; ++r) {
            hole_at += r < part ? s_each[1][r] : 0;
            src_at += r < part ? s_each[2][r] : 0;
            moved += s_each[1][r];
        }
    }
    if (nh + nsrc > 0) {                                             // a warp without any has nothing to write
        keys.marked(len, changes, [&](int n, uint32_t m) {
            const uint32_t bm = below(n), mh = m & bm, ms = m & ~bm;
            if ((mh >> lane) & 1) holes[hole_at + __popc(mh & lower)] = n;
            if ((ms >> lane) & 1) sources[src_at + __popc(ms & lower)] = n;
            hole_at += __popc(mh);
            src_at += __popc(ms);
        });
    }
    if constexpr (!FUSED) {
        if (tid == 0 && part == 0) a.ws[bh] = moved;
    } else {
        __syncthreads();                                             // the lists and the copies above are this CTA's own
        constexpr int NL = FUSED_D / 8;
        const int piece = tid % NL;
        for (int i = tid / NL; i < moved; i += NT / NL) {
            const size_t to = row + holes[i], from = row + sources[i];
            const uint4 kw = *reinterpret_cast<const uint4 *>(a.k + from * FUSED_D + piece * 8);
            const uint4 vw = *reinterpret_cast<const uint4 *>(a.v + from * FUSED_D + piece * 8);
            *reinterpret_cast<uint4 *>(a.k + to * FUSED_D + piece * 8) = kw;
            *reinterpret_cast<uint4 *>(a.v + to * FUSED_D + piece * 8) = vw;
            if (piece == 0) a.score_out[to] = a.score_in[from];
            if (piece == 1) a.pos_out[to] = a.pos_in[from];
        }
        write_len();
    }
}

// Rows of the moved tokens, their scores and positions; and the new lengths (the selection reads the old ones,
// which may be the same memory).  D / 8 lanes move a 16-byte piece each of a key row and a value row; everything that a
// thread moves is loaded before its first store (one row after the other, its score behind its key: 44 us where this
// takes 41, 32768 slots to 4096).
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 32;                                        // per CTA

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
    constexpr int NL = D / 8;
    constexpr int PER = kMoveThreads / NL;                           // rows in flight per CTA round
    const int bh = blockIdx.y, b = bh / a.Hkv;
    grid_wait();
    if (blockIdx.x == 0 && bh % a.Hkv == 0 && threadIdx.x == 0)
        a.lens_out[b] = min(min(max(a.lens_in[b], 0), a.max_len), a.budget);
    const int moved = a.ws[bh];
    const int32_t *holes = a.ws + (size_t)a.B * a.Hkv + (size_t)bh * 2 * a.cap, *sources = holes + a.cap;
    const size_t row = (size_t)bh * a.Nmax;
    const int lane = threadIdx.x % NL;
    constexpr int IT = kMoveRows / PER;
    const int i0 = blockIdx.x * kMoveRows + threadIdx.x / NL;
    if (i0 >= moved) return;
    size_t to[IT], from[IT];
    uint4 kw[IT], vw[IT];
    int x[IT];
#pragma unroll
    for (int j = 0; j < IT; ++j) {                                   // rows past the last: the first again, not written
        const int i = i0 + j * PER < moved ? i0 + j * PER : i0;
        to[j] = row + holes[i];
        from[j] = row + sources[i];
    }
#pragma unroll
    for (int j = 0; j < IT; ++j) {
        kw[j] = *reinterpret_cast<const uint4 *>(a.k + from[j] * D + lane * 8);
        vw[j] = *reinterpret_cast<const uint4 *>(a.v + from[j] * D + lane * 8);
        x[j] = lane == 0 ? __float_as_int(a.score_in[from[j]]) : lane == 1 ? a.pos_in[from[j]] : 0;
    }
#pragma unroll
    for (int j = 0; j < IT; ++j) {
        if (i0 + j * PER >= moved) break;
        *reinterpret_cast<uint4 *>(a.k + to[j] * D + lane * 8) = kw[j];
        *reinterpret_cast<uint4 *>(a.v + to[j] * D + lane * 8) = vw[j];
        if (lane == 0) a.score_out[to[j]] = __int_as_float(x[j]);
        if (lane == 1) a.pos_out[to[j]] = x[j];
    }
}

int evict_cap(int max_len, int budget) {
    const int over = max_len > budget ? max_len - budget : 0;
    return over < budget ? over : budget;
}

}  // namespace

// One launch where a head moves at most kFusedRows rows of a short row (a step's eviction: a CTA moves them while others
// still select) and a cluster can hold a sequence's heads: the lengths are written behind its barrier.  It needs no
// workspace.
constexpr int kFusedRows = 256;                                      // their lists fit into the kernel's list
constexpr int kShortRow = 2560, kClusterHeads = 16;                  // 16: more than 8 have to be asked for
static_assert(2 * kFusedRows <= kList, "moved rows' lists");
static bool fused_evict(int Hkv, int max_len, int budget) {
    return max_len <= kShortRow && evict_cap(max_len, budget) <= kFusedRows && Hkv <= kClusterHeads;
}

size_t evict_ws_bytes(int B, int Hkv, int max_len, int budget) {
    if (fused_evict(Hkv, max_len, budget)) return 0;
    return (size_t)B * Hkv * (1 + 2 * (size_t)evict_cap(max_len, budget)) * sizeof(int32_t);
}

template <int NT, typename Keys, int FUSED_D, int CL>
static cudaError_t launch_select(const EvictArgs &a, cudaStream_t s) {
    auto kern = evict_select_kernel<NT, Keys, FUSED_D, CL>;
    const bool heads = FUSED_D > 0 && a.lens_out == a.lens_in;       // a cluster of the sequence's heads
    if (heads && a.Hkv > 8) {
        const cudaError_t e = allow_large_clusters((const void *)kern);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.B * a.Hkv * CL);
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = CL > 1 ? CL : a.Hkv;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = CL > 1 || heads ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

// A row is a budget and a little more, and budgets tend to be powers of two: register capacities a quarter above those.
// One CTA's instructions bound a long row (32768 slots on one CTA: 43 us), so it is shared out.
template <int FUSED_D>
static cudaError_t launch_short(const EvictArgs &a, cudaStream_t s) {
    return a.max_len <= 1280 ? launch_select<256, RegKeys<256, 5>, FUSED_D, 1>(a, s)
                             : launch_select<256, RegKeys<256, 10>, FUSED_D, 1>(a, s);
}

static cudaError_t launch_long(const EvictArgs &a, cudaStream_t s) {
    if (a.max_len <= 5120) return launch_select<256, RegKeys<256, 10>, 0, 2>(a, s);
    if (a.max_len <= 10240) return launch_select<256, RegKeys<256, 10>, 0, 4>(a, s);
    if (a.max_len <= 20480) return launch_select<256, RegKeys<256, 10>, 0, 8>(a, s);
    if (a.max_len <= 40960) return launch_select<512, RegKeys<512, 10>, 0, 8>(a, s);
    return launch_select<512, MemKeys<512>, 0, 8>(a, s);
}

cudaError_t launch_evict(const EvictArgs &args, cudaStream_t s) {
    EvictArgs a = args;
    a.cap = evict_cap(a.max_len, a.budget);
    if (fused_evict(a.Hkv, a.max_len, a.budget))
        return a.D == 128 ? launch_short<128>(a, s) : launch_short<64>(a, s);
    const cudaError_t e = a.max_len <= kShortRow ? launch_short<0>(a, s) : launch_long(a, s);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((a.cap + kMoveRows - 1) / kMoveRows > 0 ? (a.cap + kMoveRows - 1) / kMoveRows : 1),
                    (unsigned)(a.B * a.Hkv));
    return launch_pdl(a.D == 128 ? evict_move_kernel<128> : evict_move_kernel<64>, grid, kMoveThreads, 0, s, a);
}

}  // namespace loopvq
