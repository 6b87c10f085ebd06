// Rebuilding of a coded cache's tiles for the shared-prefix attention kernels: tokens of one (layer, loop step,
// sequence, KV head) from index words through the slices, keys rotated at their positions, into shared memory as the
// products read them.
#pragma once

#include "decode_kernel.cuh"
#include "tcgen05.cuh"

namespace loopvq {

// Rows n (128 bytes of 64 channels) of a panel: 16-byte chunk j lies at chunk j ^ (n & 7).
__device__ __forceinline__ uint32_t sw128(int n, int chunk) { return (uint32_t)n * 128u + ((uint32_t)(chunk ^ (n & 7)) << 4); }

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

// A slice in shared memory: each 8-bit code's entry fills a row of 64 bytes with copies of itself, one for every second
// lane that a wavefront serves, so that two lanes at most meet in a bank, and they only for codes of equal parity (1.5
// wavefronts where one copy takes 3; rows of 128 bytes take 1, but their memory is a third stage of tiles).
constexpr int kTableBytes = 256 * 64;

struct RebuildArgs {
    const uint32_t *idx;             // index words of the KV head
    const uint16_t *slk, *slv;       // its slices
    const float *rope;
    const unsigned char *table;      // both slices in shared memory (not with one codebook per channel group)
    const unsigned char *turn;       // rope row 64 in shared memory
    uint32_t stages;                 // shared address of the stages: K upper part, K lower part, V
    uint32_t kfull, vfull, kempty, vempty;   // first barriers of the stages
    int K;
    uint64_t wait_ns;
    volatile int *dead;
};

// Fills both tables (every thread of the CTA takes part).
template <int C>
__device__ __forceinline__ void fill_tables(unsigned char *table, const uint16_t *slk, const uint16_t *slv, int K,
                                            int threads) {
#pragma unroll 4
    for (int it = threadIdx.x; it < 2 * 256 * 4; it += threads) {    // 16-byte pieces of the copies' rows
        const int kv = it / 1024, e = it / 4 % 256, slot = it % 4;
        const uint16_t *src = kv ? slv : slk;
        uint4 v = make_uint4(0, 0, 0, 0);                            // entries past K: zeros
        if (e < K) {
            if constexpr (C == 4) {
                const uint2 x = *reinterpret_cast<const uint2 *>(src + e * 4);
                v = make_uint4(x.x, x.y, x.x, x.y);
            } else {
                v = *reinterpret_cast<const uint4 *>(src + e * C + slot % (C / 8) * 8);
            }
        }
        *reinterpret_cast<uint4 *>(table + kv * kTableBytes + e * 64 + slot * 16) = v;
    }
}

// The keys of tiles 0 .. ntiles-1 of 64 tokens from tok_first, through a ring of ST stages; rw: this warp's place among
// the 8 that rebuild keys.  False: a wait ran out.
//
// A warp takes 8 tokens of the tile, a lane one token and one piece of 8 + 8 channels (8 RoPE pairs) at a time.  The 8
// lanes of a 16-byte wavefront are tokens n and n ^ 4 by 4 pieces: their chunks of the swizzled rows lie in different
// banks.  cos and sin turn from tile to tile by the fixed angle of 64 positions (4 flops a pair, where a row of the table
// per token would be 512 bytes from L2); every 8th tile they are read from the table again, so that no more than 8
// roundings add up.
//
// What bounds it is latency: a warp's visit to a tile is a chain of a wait, gathers, a rotation, stores, a fence and an
// arrival, of about the same length for one unit of work as for two.  So values have warps of their own (below), and
// index words come from a running pointer, two tiles ahead.
template <int C>
__device__ __forceinline__ uint32_t entry_copy(int lane) {           // a lane's copy of an entry, in bytes
    const int pl = lane & 3;
    // C = 4: 8 copies of 8 bytes; else 64 / (2 C) copies of C / 8 pieces of 16 bytes
    return C == 4 ? (lane & 7) * 8 : C == 32 ? pl * 16 : (C == 8 ? lane & 3 : pl) * 16;
}

// 8 channels of a piece (half 0: the low channels, 1: their partners) from the codes of its words.
template <int D, int C, bool PG>
__device__ __forceinline__ uint4 gather_piece(const RebuildArgs &b, const unsigned char *tab, const uint16_t *gsl, int sh,
                                              int half, int piece, uint32_t w0, uint32_t w1) {
    constexpr int NP = D / (2 * C);
    if constexpr (C == 4) {
        const int c0 = (w0 >> sh) & 255, c1 = (w1 >> sh) & 255;
        uint2 x, y;
        if constexpr (PG) {
            const int grp = half * NP + piece * 2;
            x = __ldg(reinterpret_cast<const uint2 *>(gsl + (size_t)min(c0, b.K - 1) * D + grp * C));
            y = __ldg(reinterpret_cast<const uint2 *>(gsl + (size_t)min(c1, b.K - 1) * D + (grp + 1) * C));
        } else {
            x = *reinterpret_cast<const uint2 *>(tab + c0 * 64);
            y = *reinterpret_cast<const uint2 *>(tab + c1 * 64);
        }
        return make_uint4(x.x, x.y, y.x, y.y);
    } else {
        const int c0 = (w0 >> sh) & 255;
        if constexpr (PG) {
            const int grp = half * NP + piece / (C / 8);
            return __ldg(reinterpret_cast<const uint4 *>(gsl + (size_t)min(c0, b.K - 1) * D + grp * C + piece % (C / 8) * 8));
        } else {
            return *reinterpret_cast<const uint4 *>(tab + c0 * 64);
        }
    }
}

template <int C>
struct Words {                                                       // index words of a piece, and words between rounds
    static constexpr int n = C == 4 ? 2 : 1;
    static constexpr int round = (C == 4 ? 8 : C == 8 ? 4 : C == 16 ? 2 : 1) * 4;
    static __device__ __forceinline__ int first(int pl) { return C == 4 ? pl * 2 : pl / (C / 8); }
};

template <int D, int C, bool PG, int ST>
__device__ __forceinline__ bool rebuild_keys(const RebuildArgs &b, int rw, int tok_first, int ntiles, int st, int len) {
    constexpr int kTile = (D / 64) * 64 * 128;
    constexpr int NP = D / (2 * C);
    constexpr int IT = D / 64;                                       // rounds of 4 pieces
    constexpr int NW = Words<C>::n;
    constexpr int kAnchor = 8;
    const int lane = threadIdx.x & 31, pl = lane & 3, tl = ((lane >> 2) & 1) * 4 + (lane >> 3);
    const unsigned char *tab = b.table + entry_copy<C>(lane);
    const float4 *turn = reinterpret_cast<const float4 *>(b.turn) + pl * 2;
    const int nl = rw * 8 + tl;
    int n = tok_first + nl;                                          // this lane's token of the tile
    const uint32_t *wp = b.idx + idx_word(n, Words<C>::first(pl), NP);
    const uint32_t lo_at = b.stages + sw128(nl, pl);                 // of round 0; a round is 4 chunks further
    const uint32_t swz = (uint32_t)(nl & 7) << 4;
    auto load_words = [&](int ahead, uint32_t (&wd)[IT][NW]) {
        const int m = n + ahead * 64;
#pragma unroll
        for (int it = 0; it < IT; ++it)
#pragma unroll
            for (int k = 0; k < NW; ++k)
                wd[it][k] = m >= st && m < len ? __ldg(wp + ahead * 64 * NP + it * Words<C>::round + k * 4) : 0u;
    };
    uint32_t wd[IT][NW], nx[IT][NW];
    load_words(0, wd);
    load_words(1, nx);
    float2 cs[IT][4], sn[IT][4];                                     // of this lane's token and channels
    int s = 0;
    uint32_t par = 1;                                                // an empty ring counts as read
    for (int t = 0; t < ntiles; ++t) {
        const bool in = n >= st && n < len;
        uint32_t n2[IT][NW];
        load_words(2, n2);                                           // two tiles ahead: a tile is shorter than a load
        if (t % kAnchor == 0) {
            const float4 *row = reinterpret_cast<const float4 *>(b.rope + (size_t)(n < len ? n : st) * D) + pl * 2;
#pragma unroll
            for (int it = 0; it < IT; ++it)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float4 c = __ldg(row + it * 8 + k), x = __ldg(row + D / 8 + it * 8 + k);
                    cs[it][2 * k] = f2(c.x, c.y);
                    cs[it][2 * k + 1] = f2(c.z, c.w);
                    sn[it][2 * k] = f2(x.x, x.y);
                    sn[it][2 * k + 1] = f2(x.z, x.w);
                }
        }
        uint4 k0[IT], k1[IT];
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const uint4 z = make_uint4(0, 0, 0, 0);
            const int piece = it * 4 + pl;
            k0[it] = in ? gather_piece<D, C, PG>(b, tab, b.slk, 0, 0, piece, wd[it][0], wd[it][NW - 1]) : z;
            k1[it] = in ? gather_piece<D, C, PG>(b, tab, b.slk, 8, 1, piece, wd[it][0], wd[it][NW - 1]) : z;
        }
        if (!__all_sync(0xffffffffu, tc::mbar_wait_or_dead(b.kempty + 8u * s, par, b.wait_ns, b.dead))) return false;
        const uint32_t off = (uint32_t)s * (3 * kTile);
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const uint32_t kl[4] = {k0[it].x, k0[it].y, k0[it].z, k0[it].w};
            const uint32_t kh[4] = {k1[it].x, k1[it].y, k1[it].z, k1[it].w};
            uint32_t ah[4], al[4], bh[4], bl[4];                     // rotated: bf16 parts of the low and high channels
            const float2 minus = f2(-1.f, -1.f);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 x = unpack2(kl[k]), y = unpack2(kh[k]), ny = unpack2(kh[k] ^ 0x80008000u);
                const float2 ra = __ffma2_rn(x, cs[it][k], __fmul2_rn(ny, sn[it][k]));
                const float2 rb = __ffma2_rn(y, cs[it][k], __fmul2_rn(x, sn[it][k]));
                ah[k] = cvt_bf16x2(ra.y, ra.x);
                bh[k] = cvt_bf16x2(rb.y, rb.x);
                const float2 da = __ffma2_rn(unpack2(ah[k]), minus, ra), db = __ffma2_rn(unpack2(bh[k]), minus, rb);
                al[k] = cvt_bf16x2(da.y, da.x);
                bl[k] = cvt_bf16x2(db.y, db.x);
            }
            // low channels 8 piece .., high channels D/2 + 8 piece ..
            const uint32_t lo = off + (it == 0 ? lo_at : b.stages + (uint32_t)nl * 128u + (((pl + 4u) << 4) ^ swz));
            const uint32_t hi = D == 128 ? lo + 64 * 128 : off + b.stages + (uint32_t)nl * 128u + (((pl + 4u) << 4) ^ swz);
            sts128(lo, make_uint4(ah[0], ah[1], ah[2], ah[3]));
            sts128(hi, make_uint4(bh[0], bh[1], bh[2], bh[3]));
            sts128(lo + kTile, make_uint4(al[0], al[1], al[2], al[3]));
            sts128(hi + kTile, make_uint4(bl[0], bl[1], bl[2], bl[3]));
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(b.kfull + 8u * s);
#pragma unroll
        for (int it = 0; it < IT; ++it)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float4 c64 = turn[it * 8 + k], s64 = turn[D / 8 + it * 8 + k];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 c = cs[it][2 * k + j], x = sn[it][2 * k + j];
                    const float2 tc2 = j ? f2(c64.z, c64.w) : f2(c64.x, c64.y);
                    const float2 ts2 = j ? f2(s64.z, s64.w) : f2(s64.x, s64.y);
                    cs[it][2 * k + j] = __ffma2_rn(c, tc2, __fmul2_rn(neg2(x), ts2));
                    sn[it][2 * k + j] = __ffma2_rn(x, tc2, __fmul2_rn(c, ts2));
                }
            }
        n += 64;
        wp += 64 * NP;
        if (++s == ST) {
            s = 0;
            par ^= 1;
        }
#pragma unroll
        for (int it = 0; it < IT; ++it)
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                wd[it][k] = nx[it][k];
                nx[it][k] = n2[it][k];
            }
    }
    return true;
}

// The values of the same tiles, by 2 warps of 32 tokens each: gathers and stores, nothing between them.
template <int D, int C, bool PG, int ST>
__device__ __forceinline__ bool rebuild_values(const RebuildArgs &b, int vw, int tok_first, int ntiles, int st, int len) {
    constexpr int kTile = (D / 64) * 64 * 128;
    constexpr int NP = D / (2 * C);
    constexpr int IT = D / 64;
    constexpr int NW = Words<C>::n;
    const int lane = threadIdx.x & 31, pl = lane & 3, tl = ((lane >> 2) & 1) * 4 + (lane >> 3);
    const unsigned char *tab = b.table + kTableBytes + entry_copy<C>(lane);
    const int n0 = vw * 32 + tl;                                     // first of this lane's tokens, 8 apart
    int n = tok_first + n0;
    const uint32_t *wp = b.idx + idx_word(n, Words<C>::first(pl), NP);
    uint32_t wd[4][IT][NW];
    auto load_words = [&]() {
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int it = 0; it < IT; ++it)
#pragma unroll
                for (int k = 0; k < NW; ++k)
                    wd[g][it][k] = n + g * 8 >= st && n + g * 8 < len
                                       ? __ldg(wp + g * 8 * NP + it * Words<C>::round + k * 4) : 0u;
    };
    load_words();
    int s = 0;
    uint32_t par = 1;
    for (int t = 0; t < ntiles; ++t) {
        if (!__all_sync(0xffffffffu, tc::mbar_wait_or_dead(b.vempty + 8u * s, par, b.wait_ns, b.dead))) return false;
        const uint32_t vb = b.stages + (uint32_t)s * (3 * kTile) + 2 * kTile;
#pragma unroll
        for (int g0 = 0; g0 < 4; g0 += 2) {                          // loads of two groups before their stores
            uint4 v[2][IT][2];
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const int m = n + (g0 + g) * 8, piece = it * 4 + pl;
                    const uint32_t w0 = wd[g0 + g][it][0], w1 = wd[g0 + g][it][NW - 1];
                    v[g][it][0] = gather_piece<D, C, PG>(b, tab, b.slv, 16, 0, piece, w0, w1);
                    v[g][it][1] = gather_piece<D, C, PG>(b, tab, b.slv, 24, 1, piece, w0, w1);
                    if (m < st || m >= len) v[g][it][0] = v[g][it][1] = make_uint4(0, 0, 0, 0);
                }
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const int nl = n0 + (g0 + g) * 8, piece = it * 4 + pl;
                    sts128(vb + sw128(nl, piece), v[g][it][0]);
                    sts128(vb + (D == 128 ? (64 * 128) + sw128(nl, piece) : sw128(nl, piece + 4)), v[g][it][1]);
                }
        }
        n += 64;
        wp += 64 * NP;
        load_words();                                                // the next tile's, under the fence and the wait
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(b.vfull + 8u * s);
        if (++s == ST) {
            s = 0;
            par ^= 1;
        }
    }
    return true;
}

}  // namespace loopvq
