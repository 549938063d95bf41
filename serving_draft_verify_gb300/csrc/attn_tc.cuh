// Attention of many query rows a request (verification of a long draft, wide groups of
// heads, prompts): 128 query rows of a key head at a time on tcgen05.
//
// At 128 rows a key costs 4 * 128 * D operations for 4 D bytes, more than the warp-level
// instructions can do while the bytes arrive, and less than tcgen05 can: per unit of 128 keys
// at D = 128 the products take about 1536 tensor cycles (S once, P V twice) and the softmax
// about as many of one warpgroup, next to 2800 cycles for the unit's 64 KB at the measured
// bandwidth.  So one block an SM, with a warp for each thing that can run by itself:
//
//   warp 0      keys into a ring of two units by TMA (boxes of up to 128 rows that lie on one page,
//               128-byte swizzle), running ahead across pieces;
//   warp 1      S = Q K^T into one of two TMEM buffers, a unit ahead;
//   warp 2      O += P V with P from TMEM and V as it lies (its rows are the contraction: an
//               MN-major operand);
//   warp 3      values like the keys, and before a piece's its queries, into the other of two buffers;
//   warps 4-11  two threads a query row, each with half of a unit's keys: P = 2^(S - m) as two
//               bf16 terms (split_bf16, so that 15 bits of P count) into TMEM, the sum, and half of
//               the output's columns at the end.
// The output in TMEM is rescaled only where a maximum has grown by more than 2^8 over the one
// in use (the factor stays in P and the sum alike until then), so the two threads of a row
// exchange their maxima in those units alone.  The instruction cache is a bound here: with six
// roles in one kernel, what runs once a piece or never (the walk, the joining, waits that have to
// wait) stands in functions of its own.
// 128 requests of up to 6000 keys, up to 17 rows, 32 heads on 8, pages of 16: 501 us for 1.65 GB (3.3
// TB/s).  What bounds it is the copying: a box cannot leave its page, and boxes of 16 rows of 128
// bytes take some 150 cycles each, 4900 cycles a unit (pages of 32 rows and more: 3800, the softmax).
// Boxes of whole rows, a softmax in two groups by turns and copies by threads were all slower.
//
// TMEM (512 columns): S 2 x 128, P 64 high + 64 low, O up to 128.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "attn_mma.cuh"
#include "engine.cuh"
#include "tc.cuh"

namespace dspark {
namespace attn {

// Shared-memory descriptor of an MN-major operand with the 128-byte swizzle: 64 elements of the
// M / N extent to a 128-byte row, a row for every k; 8 rows 1024 bytes apart (stride), the next 64
// elements `half` bytes apart (leading).
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t half) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((half >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}
// D[tmem] (+)= A[tmem] B[smem desc].
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// 32 consecutive TMEM columns of this warp's lanes from every k-th of v.
template <int k>
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(__float_as_uint(v[0 * k])), "r"(__float_as_uint(v[1 * k])), "r"(__float_as_uint(v[2 * k])),
        "r"(__float_as_uint(v[3 * k])), "r"(__float_as_uint(v[4 * k])), "r"(__float_as_uint(v[5 * k])),
        "r"(__float_as_uint(v[6 * k])), "r"(__float_as_uint(v[7 * k])), "r"(__float_as_uint(v[8 * k])),
        "r"(__float_as_uint(v[9 * k])), "r"(__float_as_uint(v[10 * k])), "r"(__float_as_uint(v[11 * k])),
        "r"(__float_as_uint(v[12 * k])), "r"(__float_as_uint(v[13 * k])), "r"(__float_as_uint(v[14 * k])),
        "r"(__float_as_uint(v[15 * k])), "r"(__float_as_uint(v[16 * k])), "r"(__float_as_uint(v[17 * k])),
        "r"(__float_as_uint(v[18 * k])), "r"(__float_as_uint(v[19 * k])), "r"(__float_as_uint(v[20 * k])),
        "r"(__float_as_uint(v[21 * k])), "r"(__float_as_uint(v[22 * k])), "r"(__float_as_uint(v[23 * k])),
        "r"(__float_as_uint(v[24 * k])), "r"(__float_as_uint(v[25 * k])), "r"(__float_as_uint(v[26 * k])),
        "r"(__float_as_uint(v[27 * k])), "r"(__float_as_uint(v[28 * k])), "r"(__float_as_uint(v[29 * k])),
        "r"(__float_as_uint(v[30 * k])), "r"(__float_as_uint(v[31 * k]))
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

constexpr int kTcM = 128, kTcKT = 128, kTcThreads = 384, kTcSoft = 256;   // kTcSoft: threads of the softmax

template <int DT>
struct TcShape {
    static constexpr int kHalves = DT / 64;
    static constexpr int kHalf = 128 * 128;                  // bytes of 64 columns of 128 rows
    static constexpr int kTile = kHalves * kHalf;
    static constexpr int kSmem = 6 * kTile + 1024;           // Q, K, V twice each; 1024: alignment
};
struct TcBars {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], q_full[2], q_empty[2], s_full[2], s_empty[2], p_full, pv_done;
};

__device__ __noinline__ bool next_piece(Walk<kTcM, kTcKT>& walk, Piece& pc) { return walk.next(pc); }
// A wait that runs out ends all waiting: every role goes on through its units without issuing
// anything, so that the block ends, and the status tells.
__device__ __noinline__ void long_wait(uint64_t* bar, uint32_t parity, volatile int* dead, StatusBlock* status) {
    if (*dead) return;
    if (!mbar_wait(bar, parity)) {
        *dead = 1;
        tell(status, DSPARK_ERR_TIMEOUT, 1);
    }
}

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool softmax_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(x ? 1u : 0u)
        : "memory");
    return r != 0;
}

template <int DT>
__global__ void __launch_bounds__(kTcThreads, 1)
    attend_tc(const __grid_constant__ Args p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, int box) {
    using Sh = TcShape<DT>;
    extern __shared__ unsigned char raw[];
    unsigned char* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    unsigned char* s_q = smem;                               // [2] tiles: [halves][128 rows][128 bytes]
    unsigned char* s_k = smem + 2 * Sh::kTile;
    unsigned char* s_v = smem + 4 * Sh::kTile;
    __shared__ long long scratch[38];
    __shared__ __align__(8) TcBars bars;
    __shared__ uint32_t s_tmem;
    __shared__ float2 s_row[kTcM];
    __shared__ float s_two[2][kTcM];                         // what the two threads of a row tell each other
    __shared__ int s_flag;
    __shared__ volatile int s_dead, s_keep;                  // s_keep: the piece's first product adds to what O holds
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.k_full[i], 1);
            mbar_init(&bars.k_empty[i], 1);
            mbar_init(&bars.v_full[i], 1);
            mbar_init(&bars.v_empty[i], 1);
            mbar_init(&bars.q_full[i], 32);
            mbar_init(&bars.q_empty[i], 1);
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.s_empty[i], kTcSoft);
        }
        mbar_init(&bars.p_full, kTcSoft);
        mbar_init(&bars.pv_done, 1);
        fence_mbar_init();
        s_dead = 0;
        s_keep = 0;
    }
    if (w == 1) tc::tmem_alloc(&s_tmem, 512);
    tc::fence_before_sync();
    const Start st = find_start<kTcM, kTcKT, kTcThreads>(p, scratch);
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem, t_p = tmem + 256, t_o = tmem + 384;

    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!mbar_try_wait(bar, parity & 1)) long_wait(bar, parity & 1, &s_dead, p.status);
    };
    Walk<kTcM, kTcKT> walk(p, st);
    Piece pc;
    uint32_t i = 0;                                          // units done

    if (w == 0 || w == 3) {
        // -------------------------------- keys; queries (a piece at a time) and values ---
        const bool keys = w == 0;
        const CUtensorMap* map = keys ? &kmap : &vmap;
        uint64_t *full = keys ? bars.k_full : bars.v_full, *empty = keys ? bars.k_empty : bars.v_empty;
        unsigned char* ring = keys ? s_k : s_v;
        const uint64_t policy = policy_evict_normal();
        const int shift = __ffs(box) - 1;                        // a box is a power of two of rows
        for (uint32_t n = 0; next_piece(walk, pc); ++n) {
            if (!keys) {
                wait(&bars.q_empty[n & 1], (n >> 1) + 1);
                const int left = pc.r.n * p.G - pc.tile * kTcM, valid = left < kTcM ? left : kTcM;
                const uint32_t to = smem_u32(s_q) + (n & 1) * Sh::kTile;
                const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
#pragma unroll 2
                for (int e = lane; e < kTcM * (DT / 8); e += 32) {
                    const int m = e / (DT / 8), c = e % (DT / 8), qi = pc.tile * kTcM + m;
                    const bool real = m < valid && c * 8 < p.D;
                    const int64_t at = real ? (static_cast<int64_t>(pc.r.row0) + qi / p.G) * p.q_stride +
                                                  static_cast<int64_t>(pc.h * p.G + qi % p.G) * p.D + c * 8
                                            : 0;
                    copy16(to + (c >> 3) * Sh::kHalf + m * 128 + (((c & 7) ^ (m & 7)) << 4), q + at, real);
                }
                cp_async_wait_all();
                fence_proxy_async_smem();
                mbar_arrive(&bars.q_full[n & 1]);
            }
            const int hi = pc.span.hi, seen = pc.span.seen, b = pc.b, h = pc.h;
            int k0 = pc.span.lo + pc.u0 * kTcKT;
#pragma unroll 1
            for (int u = pc.u0; u < pc.u1; ++u, ++i, k0 += kTcKT) {
                // boxes wholly before the first key that the tile sees stay away: the softmax makes those
                // values 0, as it does those past the last key
                const int stage = i & 1, before = max(seen - k0, 0) >> shift, boxes = ((min(kTcKT, hi - k0) + box - 1) >> shift) - before;
                // lane l finds the row of box l; lane 0 issues them all (an instruction that several
                // lanes issue goes lane by lane, at several times the cost)
                int y = 0;
                if (lane < boxes) {
                    const int key = k0 + (before + lane) * box, blk = key / p.page;
                    y = (page_id(p, b, blk) * p.Hkv + h) * p.page + (key - blk * p.page);
                }
                if (lane == 0) {
                    wait(&empty[stage], (i >> 1) + 1);
                    if (!s_dead) mbar_arrive_expect_tx(&full[stage], boxes * box * 128 * Sh::kHalves);
                }
                unsigned char* to = ring + stage * Sh::kTile + before * box * 128;
#pragma unroll 1
                for (int j = 0; j < boxes; ++j, to += box * 128) {
                    const int yj = __shfl_sync(0xffffffffu, y, j);
                    if (lane == 0 && !s_dead)
#pragma unroll
                        for (int c = 0; c < Sh::kHalves; ++c)
                            tc::tma_load_2d(to + c * Sh::kHalf, map, 64 * c, yj, &full[stage], policy);
                }
            }
        }
        // where a wait ran out, copies still in flight end before the block does
        if (s_dead && lane == 0)
            for (uint32_t j = i > 2 ? i - 2 : 0; j < i; ++j) mbar_wait(&full[j & 1], (j >> 1) & 1);
        __syncwarp();
    } else if (w == 1) {
        // ---------------------------------------------------------------- scores ---
        if (lane == 0) {
            constexpr uint32_t id_s = tc::idesc_bf16_f32(kTcM, kTcKT);
            for (uint32_t n = 0; next_piece(walk, pc); ++n) {
                const uint32_t qa = smem_u32(s_q) + (n & 1) * Sh::kTile;
                wait(&bars.q_full[n & 1], n >> 1);
#pragma unroll 1
                for (int u = pc.u1 - pc.u0; u > 0; --u, ++i) {
                    const int stage = i & 1;
                    const uint32_t ka = smem_u32(s_k) + stage * Sh::kTile;
                    wait(&bars.s_empty[stage], (i >> 1) + 1);
                    wait(&bars.k_full[stage], i >> 1);
                    tc::fence_after_sync();
                    if (s_dead) continue;
#pragma unroll
                    for (int ks = 0; ks < DT / 16; ++ks) {
                        const uint32_t off = (ks >> 2) * Sh::kHalf + (ks & 3) * 32;
                        tc::mma_bf16(tmem + stage * 128, tc::smem_desc_sw128(qa + off), tc::smem_desc_sw128(ka + off), id_s, ks > 0);
                    }
                    tc::commit(&bars.s_full[stage]);
                    tc::commit(&bars.k_empty[stage]);
                    if (u == 1) tc::commit(&bars.q_empty[n & 1]);
                }
            }
        }
        __syncwarp();
    } else if (w == 2) {
        // ---------------------------------------------------------------- output ---
        if (lane == 0) {
            constexpr uint32_t id_o = tc::idesc_bf16_f32(kTcM, DT) | (1u << 16);      // B is MN-major
            while (next_piece(walk, pc)) {
                const int n = pc.u1 - pc.u0;
#pragma unroll 1
                for (int u = 0; u < n; ++u, ++i) {
                    const int stage = i & 1;
                    const uint64_t vd = desc_mn_sw128(smem_u32(s_v) + stage * Sh::kTile, Sh::kHalf);
                    wait(&bars.v_full[stage], i >> 1);
                    wait(&bars.p_full, i);
                    tc::fence_after_sync();
                    if (s_dead) continue;
                    const bool keep = u > 0 || s_keep;
                    // 16 keys a step: 2048 bytes on in V, 8 columns on in P (the high terms, then the low)
#pragma unroll
                    for (int ks = 0; ks < kTcKT / 8; ++ks)
                        mma_bf16_ts(t_o, t_p + ks * 8, vd + (ks & 7) * (2048 >> 4), id_o, keep || ks > 0);
                    tc::commit(&bars.pv_done);
                    tc::commit(&bars.v_empty[stage]);
                }
            }
        }
        __syncwarp();
    } else {
        // --------------------------------------------------------------- softmax ---
        const int m = (tid - 128) & 127, half = (tid - 128) >> 7;   // the query row (TMEM lane), the half of the keys
        const uint32_t lanes = static_cast<uint32_t>(w & 3) << 21;  // (warp's first lane) << 16
        constexpr int kCols = DT / 2, kKeys = kTcKT / 2;
        const int d0 = half * kCols;                                // first of the thread's output columns
        const float ninf = -__uint_as_float(0x7f800000u);
        while (next_piece(walk, pc)) {
            float used = ninf, l = 0.f;
            const int left = pc.r.n * p.G - pc.tile * kTcM, valid = left < kTcM ? left : kTcM;
            const bool busy = (w & 3) * 32 < valid;                     // the warp has rows
            const int pos = pc.r.len + (pc.tile * kTcM + m) / p.G;      // the row's position, the tile's first and last
            const int pos_lo = pc.r.len + pc.tile * kTcM / p.G, pos_hi = pc.span.hi - 1;
            const int n = pc.u1 - pc.u0;
            int k0 = pc.span.lo + pc.u0 * kTcKT;
            if (tid == 128) s_keep = 0;
#pragma unroll 1
            for (int u = 0; u < n; ++u, ++i, k0 += kTcKT) {
                const int stage = i & 1;
                const bool first = u == 0;
                const bool masked = k0 + kTcKT - 1 > pos_lo || (p.window > 0 && k0 <= pos_hi - p.window);
                int c_lo = 0, c_hi = kTcKT;                             // the columns of this unit that the row sees
                if (masked) {
                    c_hi = min(min(pos, pos_hi) + 1 - k0, kTcKT);
                    if (p.window > 0) c_lo = max(pos - p.window + 1 - k0, 0);
                    // Values at keys past the last one or before the first, and values that are not finite at
                    // keys that only some rows see, must not meet the product (0 times them is not 0).  The
                    // former become 0; the latter are added here to the rows that see them and become 0 too.
                    wait(&bars.v_full[stage], i >> 1);
                    unsigned char* v = s_v + stage * Sh::kTile;
                    bool odd = false;
                    if (half < Sh::kHalves) {
                        uint4* x = reinterpret_cast<uint4*>(v + half * Sh::kHalf + m * 128);
                        if (k0 + m > pos_hi || k0 + m < pc.span.seen) {
#pragma unroll
                            for (int c = 0; c < 8; ++c) x[c] = make_uint4(0, 0, 0, 0);
                        } else {
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                odd |= any_odd<false>(x[c].x) || any_odd<false>(x[c].y) || any_odd<false>(x[c].z) || any_odd<false>(x[c].w);
                        }
                    }
                    const bool some = softmax_any(odd);
                    if (first && tid == 128 && some) s_keep = 1;
                    if (some) {
                        if (i > 0) wait(&bars.pv_done, i - 1);
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int c = d0; c < d0 + kCols; c += 32) {
                            float o[32];
                            if (first) {
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] = 0.f;
                            } else {
                                tc::tmem_ld32(t_o + lanes + c, o);
                                tc::tmem_ld_wait();
                            }
#pragma unroll 1
                            for (int j = c_lo; j < c_hi; ++j) {
                                const unsigned char* at = v + (c >> 6) * Sh::kHalf + j * 128;
#pragma unroll
                                for (int k = 0; k < 32; ++k) {
                                    const int d = (c & 63) + k;
                                    const uint32_t bits = *reinterpret_cast<const uint16_t*>(at + (((d >> 3) ^ (j & 7)) << 4) + (d & 7) * 2);
                                    if (any_odd<false>(bits)) o[k] += bf16lo(bits);
                                }
                            }
                            __syncwarp();
                            tmem_st32<1>(t_o + lanes + c, o);
                        }
                        tmem_st_wait();
                        softmax_sync();
                        if (half < Sh::kHalves)
                            for (int c = 0; c < 32; ++c) {
                                uint32_t* x = reinterpret_cast<uint32_t*>(v + half * Sh::kHalf + m * 128) + c;
                                *x = without_odd<false>(*x);
                            }
                    }
                    fence_proxy_async_smem();
                }
                wait(&bars.s_full[stage], i >> 1);
                tc::fence_after_sync();
                float s[kKeys];
                float top = ninf;
                if (busy) {
                    tc::tmem_ld32(tmem + stage * 128 + lanes + half * kKeys, s);
                    tc::tmem_ld32(tmem + stage * 128 + lanes + half * kKeys + 32, s + 32);
                    tc::tmem_ld_wait();
                    if (masked) {
                        c_lo -= half * kKeys;
                        c_hi -= half * kKeys;
#pragma unroll
                        for (int c = 0; c < kKeys; ++c)
                            if (c < c_lo || c >= c_hi) s[c] = ninf;
                    }
                    float t4[4] = {ninf, ninf, ninf, ninf};
#pragma unroll
                    for (int c = 0; c < kKeys; ++c) t4[c & 3] = fmaxf(t4[c & 3], s[c]);
                    top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * p.scale_log2;
                }
                tc::fence_before_sync();
                mbar_arrive(&bars.s_empty[stage]);
                if (softmax_any(first || top > used + 8.f)) {
                    s_two[half][m] = top;
                    softmax_sync();
                    const float next = fmaxf(used, fmaxf(s_two[0][m], s_two[1][m]));
                    if (!first) {
                        const float a = fast_exp2(used - (next == ninf ? 0.f : next));
                        wait(&bars.pv_done, i - 1);
                        tc::fence_after_sync();
                        if (busy) {
#pragma unroll 1
                            for (int c = d0; c < d0 + kCols; c += 32) {
                                float o[32];
                                tc::tmem_ld32(t_o + lanes + c, o);
                                tc::tmem_ld_wait();
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] *= a;
                                tmem_st32<1>(t_o + lanes + c, o);
                            }
                            tmem_st_wait();
                        }
                        l *= a;
                    }
                    used = next;
                }
                if (busy) {
                    const float use = used == ninf ? 0.f : used;
                    float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < kKeys; c += 2) {
                        const float e0 = fast_exp2(fmaf(s[c], p.scale_log2, -use)), e1 = fast_exp2(fmaf(s[c + 1], p.scale_log2, -use));
                        l4[c & 2] += e0;
                        l4[(c & 2) + 1] += e1;
                        // the two terms of both take the scores' places: high, then low
                        uint32_t high, low;
                        split_bf16(e0, e1, high, low);
                        s[c] = __uint_as_float(high);
                        s[c + 1] = __uint_as_float(low);
                    }
                    l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
                }
                if (i > 0) wait(&bars.pv_done, i - 1);                  // the last product has read P
                tc::fence_after_sync();
                if (busy) {
                    tmem_st32<2>(t_p + lanes + half * 32, s);
                    tmem_st32<2>(t_p + lanes + 64 + half * 32, s + 1);
                    tmem_st_wait();
                }
                tc::fence_before_sync();
                mbar_arrive(&bars.p_full);
            }
            // ---- the piece is done: its rows out of TMEM
            s_two[half][m] = l;
            wait(&bars.pv_done, i - 1);
            tc::fence_after_sync();
            softmax_sync();
            l = s_two[0][m] + s_two[1][m];
            const bool whole = pc.whole(), mine = m < valid;
            const int qi = pc.tile * kTcM + m, head = pc.h * p.G + qi % p.G;
            const int64_t row = static_cast<int64_t>(pc.r.row0) + qi / p.G;
            const int64_t at = part_place(blockIdx.x, pc.u0 == 0) * kTcM + m;
            const float inv = l != 0.f ? 1.f / l : 0.f;
            if (busy) {
#pragma unroll 1
                for (int c = d0; c < d0 + kCols; c += 32) {
                    float o[32];
                    tc::tmem_ld32(t_o + lanes + c, o);
                    tc::tmem_ld_wait();
                    if (mine && whole) {
                        __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + (row * p.Hq + head) * p.D + c;
#pragma unroll
                        for (int k = 0; k < 32; k += 8) {
                            if (c + k >= p.D) break;
                            uint4 x = make_uint4(0, 0, 0, 0);
                            if (l != 0.f)
                                x = make_uint4(pack_bf16(o[k] * inv, o[k + 1] * inv), pack_bf16(o[k + 2] * inv, o[k + 3] * inv),
                                               pack_bf16(o[k + 4] * inv, o[k + 5] * inv), pack_bf16(o[k + 6] * inv, o[k + 7] * inv));
                            *reinterpret_cast<uint4*>(to + k) = x;
                        }
                    } else if (mine) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            if (c + k >= p.D) break;
                            *reinterpret_cast<float4*>(p.part_o + at * p.D + c + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                        }
                    }
                    __syncwarp();
                }
                if (mine && half == 0) {
                    if (!whole) reinterpret_cast<float2*>(p.part_ml)[at] = make_float2(used, l);
                    else if (p.lse != nullptr) p.lse[row * p.Hq + head] = lse_of(used, l);
                }
            }
            tc::fence_before_sync();
            if (!whole && part_done(p, pc, st, &s_flag, tid - 128, [] { softmax_sync(); }))
                join_parts<__nv_bfloat16, kTcM, kTcSoft>(p, pc, st, s_row, tid - 128, [] { softmax_sync(); });
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (w == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
    if (blockIdx.x == 0) head_cleared();
}

// Rows of a TMA box: the largest power of two that divides the page, so that a box lies on one
// page and units (multiples of 128 keys) start on a box.
inline int tc_box(int page) {
    const int b = page & -page;
    return b < 128 ? b : 128;
}
// Whether the caches can be read so: 64 columns to a box, 8 rows are the swizzle's period, and
// rows are counted in 32 bits.  The largest score is found before scaling: the scale is positive.
inline bool tc_fits(const Args& p) {
    return p.scale_log2 > 0.f && p.D >= 64 && p.D <= 128 && tc_box(p.page) >= 8 && static_cast<int64_t>(p.num_blocks) * p.Hkv * p.page <= 0x7fffffffll;
}
inline bool encode_cache(CUtensorMap* map, const void* cache, const Args& p, int box) {
    auto enc = eng::tensor_map_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.D), static_cast<cuuint64_t>(p.num_blocks) * p.Hkv * p.page};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.D) * 2};
    const cuuint32_t size[2] = {64, static_cast<cuuint32_t>(box)};
    const cuuint32_t step[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(cache), dims, strides, size, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DT>
dspark_status_t launch_tc(const Args& p, cudaStream_t s) {
    static OncePerDevice once;
    const int dev = current_device();
    if (once.run(dev, [] {
            return cudaFuncSetAttribute(attend_tc<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcShape<DT>::kSmem);
        }) != cudaSuccess)
        return DSPARK_ERR_CUDA;
    CUtensorMap km, vm;
    const int box = tc_box(p.page);
    if (!encode_cache(&km, p.kc, p, box) || !encode_cache(&vm, p.vc, p, box)) return DSPARK_ERR_CUDA;
    const int grid = grid_for(sm_count(dev), kTcM);
    if (grid < 1) return DSPARK_ERR_CUDA;
    return launch_cleared(p.status, kHeadBytes, attend_tc<DT>, dim3(grid), kTcThreads, TcShape<DT>::kSmem, s, p, km, vm, box);
}

}  // namespace attn
}  // namespace dspark
