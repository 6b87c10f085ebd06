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
// wavefronts where one copy takes 3; rows of 128 bytes take 1, but their memory is a fourth stage of tiles: 32768 x 32
// queries, 8 channels per code, 71 us against 78).
constexpr int kTableBytes = 256 * 64;

struct RebuildArgs {
    const uint32_t *idx;             // index words of the KV head
    const uint16_t *slk, *slv;       // its slices
    const float *rope;
    const unsigned char *table;      // both slices in shared memory (not with one codebook per channel group)
    const unsigned char *turn;       // rope row 64 in shared memory
    uint32_t stages;                 // shared address of the stages: KP bf16 parts of K from the upper one on, V
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
// the 8 that rebuild keys; KP: bf16 parts of a key (2 leave 2^-17 of it, 3 all of an fp32 value).  False: a wait ran out.
//
// A lane takes one piece of 8 + 8 channels (8 RoPE pairs) of a token, a warp 4 pieces of 8 tokens, and at D = 128 of the 8
// tokens 32 further on.  The 8 lanes of a 16-byte wavefront are tokens n and n ^ 4 by 4 pieces: their chunks of the
// swizzled rows lie in different banks.  cos and sin turn from tile to tile by the fixed angle of 64 positions (4 flops a
// pair, where a row of the table per token would be 512 bytes from L2), whose own cosines and sines are the same for both
// tokens and stay in registers; every 8th tile the table is read again, so that no more than 8 roundings add up.
//
// What bounds it is the shared-memory pipe (gathers, stores and the products' operands: 86% busy), and before that the
// latency of a warp's visit to a tile: so values have warps of their own (below), and index words come from a running
// pointer, two tiles ahead.  16 warps with one token a lane were no faster (76.8 us where 8 took 73.5, 32768 x 32).
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

template <int D, int C, bool PG, int ST, int KP>
__device__ __forceinline__ bool rebuild_keys(const RebuildArgs &b, int rw, int tok_first, int ntiles, int st, int len) {
    constexpr int kTile = (D / 64) * 64 * 128;
    constexpr int NP = D / (2 * C);
    constexpr int U = D / 64;                                        // tokens per lane, 32 apart
    constexpr int NW = Words<C>::n;
    constexpr int kAnchor = 8;
    const int lane = threadIdx.x & 31, pl = lane & 3, tl = ((lane >> 2) & 1) * 4 + (lane >> 3);
    const int round = rw % U, piece = round * 4 + pl;                // low channels 8 piece .., high ones D/2 + 8 piece ..
    const unsigned char *tab = b.table + entry_copy<C>(lane);
    const int nl = (rw / U) * 8 + tl;
    int n = tok_first + nl;                                          // this lane's first token of the tile
    const uint32_t *wp = b.idx + idx_word(n, Words<C>::first(pl), NP) + round * Words<C>::round;
    const uint32_t lo_at = b.stages + sw128(nl, piece);
    const uint32_t hi_at = D == 128 ? lo_at + 64 * 128 : b.stages + sw128(nl, piece + 4);
    auto load_words = [&](int ahead, uint32_t (&wd)[U][NW]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int m = n + ahead * 64 + u * 32;
#pragma unroll
            for (int k = 0; k < NW; ++k)
                wd[u][k] = m >= st && m < len ? __ldg(wp + (ahead * 64 + u * 32) * NP + k * 4) : 0u;
        }
    };
    uint32_t wd[U][NW], nx[U][NW];
    load_words(0, wd);
    load_words(1, nx);
    float2 cs[U][4] = {}, sn[U][4] = {};                             // of this lane's tokens and channels
    float2 tc64[4], ts64[4];                                         // of the turn by 64 positions
    {
        const float4 *turn = reinterpret_cast<const float4 *>(b.turn) + piece * 2;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float4 c = turn[k], x = turn[D / 8 + k];
            tc64[2 * k] = f2(c.x, c.y);
            tc64[2 * k + 1] = f2(c.z, c.w);
            ts64[2 * k] = f2(x.x, x.y);
            ts64[2 * k + 1] = f2(x.z, x.w);
        }
    }
    int s = 0;
    uint32_t par = 1;                                                // an empty ring counts as read
    for (int t = 0; t < ntiles; ++t) {
        uint32_t n2[U][NW];
        load_words(2, n2);                                           // two tiles ahead: a tile is shorter than a load
        if (t % kAnchor == 0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int m = n + u * 32;
                const float4 *row = reinterpret_cast<const float4 *>(b.rope + (size_t)(m < len ? m : st) * D) + piece * 2;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float4 c = __ldg(row + k), x = __ldg(row + D / 8 + k);
                    cs[u][2 * k] = f2(c.x, c.y);
                    cs[u][2 * k + 1] = f2(c.z, c.w);
                    sn[u][2 * k] = f2(x.x, x.y);
                    sn[u][2 * k + 1] = f2(x.z, x.w);
                }
            }
        }
        uint4 k0[U], k1[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int m = n + u * 32;
            k0[u] = k1[u] = make_uint4(0, 0, 0, 0);
            if (m >= st && m < len) {
                k0[u] = gather_piece<D, C, PG>(b, tab, b.slk, 0, 0, piece, wd[u][0], wd[u][NW - 1]);
                k1[u] = gather_piece<D, C, PG>(b, tab, b.slk, 8, 1, piece, wd[u][0], wd[u][NW - 1]);
            }
        }
        if (!__all_sync(0xffffffffu, tc::mbar_wait_or_dead(b.kempty + 8u * s, par, b.wait_ns, b.dead))) return false;
        const uint32_t off = (uint32_t)s * ((KP + 1) * kTile);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t kl[4] = {k0[u].x, k0[u].y, k0[u].z, k0[u].w};
            const uint32_t kh[4] = {k1[u].x, k1[u].y, k1[u].z, k1[u].w};
            uint32_t ah[4], al[4], bh[4], bl[4];                     // rotated: bf16 parts of the low and high channels
            [[maybe_unused]] uint32_t az[4], bz[4];                  // third ones
            const float2 minus = f2(-1.f, -1.f);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 x = unpack2(kl[k]), y = unpack2(kh[k]), ny = unpack2(kh[k] ^ 0x80008000u);
                const float2 ra = __ffma2_rn(x, cs[u][k], __fmul2_rn(ny, sn[u][k]));
                const float2 rb = __ffma2_rn(y, cs[u][k], __fmul2_rn(x, sn[u][k]));
                ah[k] = cvt_bf16x2(ra.y, ra.x);
                bh[k] = cvt_bf16x2(rb.y, rb.x);
                const float2 da = __ffma2_rn(unpack2(ah[k]), minus, ra), db = __ffma2_rn(unpack2(bh[k]), minus, rb);
                al[k] = cvt_bf16x2(da.y, da.x);
                bl[k] = cvt_bf16x2(db.y, db.x);
                if constexpr (KP == 3) {
                    const float2 ea = __ffma2_rn(unpack2(al[k]), minus, da), eb = __ffma2_rn(unpack2(bl[k]), minus, db);
                    az[k] = cvt_bf16x2(ea.y, ea.x);
                    bz[k] = cvt_bf16x2(eb.y, eb.x);
                }
            }
            const uint32_t at = off + u * (32 * 128);                // 32 rows further: the same swizzle
            sts128(lo_at + at, make_uint4(ah[0], ah[1], ah[2], ah[3]));
            sts128(hi_at + at, make_uint4(bh[0], bh[1], bh[2], bh[3]));
            sts128(lo_at + at + kTile, make_uint4(al[0], al[1], al[2], al[3]));
            sts128(hi_at + at + kTile, make_uint4(bl[0], bl[1], bl[2], bl[3]));
            if constexpr (KP == 3) {
                sts128(lo_at + at + 2 * kTile, make_uint4(az[0], az[1], az[2], az[3]));
                sts128(hi_at + at + 2 * kTile, make_uint4(bz[0], bz[1], bz[2], bz[3]));
            }
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(b.kfull + 8u * s);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 c = cs[u][k], x = sn[u][k];
                cs[u][k] = __ffma2_rn(c, tc64[k], __fmul2_rn(neg2(x), ts64[k]));
                sn[u][k] = __ffma2_rn(x, tc64[k], __fmul2_rn(c, ts64[k]));
            }
        n += 64;
        wp += 64 * NP;
        if (++s == ST) {
            s = 0;
            par ^= 1;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                wd[u][k] = nx[u][k];
                nx[u][k] = n2[u][k];
            }
    }
    return true;
}

// The values of the same tiles, by 2 warps of 32 tokens each: gathers and stores, nothing between them.
template <int D, int C, bool PG, int ST, int KP>
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
        const uint32_t vb = b.stages + (uint32_t)s * ((KP + 1) * kTile) + KP * kTile;
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
