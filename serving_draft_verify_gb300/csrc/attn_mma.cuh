// Attention of few query rows a request (plain decoding, short drafts): 16 query rows of a
// key head at a time on the warp-level tensor instructions (tiles of 32 rows held twice the
// registers and were slower than two tiles of 16 wherever both were measured).
//
// Bound by the cache's bytes, so the kernel is built around keeping loads in flight.
// The four warps of a block share nothing in the loop: warp w takes keys w KS .. w KS + KS - 1
// of every unit of 4 KS, with a ring of its own for them (asynchronous 16-byte copies,
// 128-byte rows swizzled by chunk ^ (row mod 8), so that ldmatrix is free of conflicts),
// its own running maximum and sum and its own rows of the output in registers.  Nothing
// waits for another warp until the piece ends and the four results join in shared memory.
//
//   S = Q K^T    m16n8k16, keys as columns; S stays in registers,
//   P = 2^(S - m), rescaling the output only in steps where a maximum moved,
//   O += P V     P's accumulator layout is the A operand's layout.
//
// Three blocks an SM (168 registers, rings of two steps of 8 KB a warp): with three steps and two
// blocks, fixed latencies left the 8-bit caches at half the speed of their bytes (64 requests of
// 4000 keys: 87 us, now 74; bf16 112 and 110, of 500 keys 100 and 87).  64 requests of up to 16384
// keys, one row each, bf16: 352 us for 2.4 GB, 6.8 TB/s, which is what a copy reaches.
//
// bf16 caches: P goes in as two bf16 terms (split_bf16: 15 bits of P at least), which costs a second
// product but no bytes.  8-bit caches: stored values are exact in f16, so both products
// run in f16; Q's rows are scaled by a power of two into f16's range, P carries a factor
// 2^14 that the sum carries too and is rounded to 11 bits (half a step of 2^-12, below the
// output's own 2^-9).  Bytes of a 16-byte chunk are taken in the order that one ldmatrix
// gives them (Q's columns are stored in that order), so a conversion is all they need.
#pragma once

#include "attn.cuh"

namespace dspark {
namespace attn {

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool kHalf>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    if constexpr (kHalf)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two 8-bit values as two f16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two weights as two bf16 terms each.  The high one is cut off, not rounded, so that the rest is never
// negative, and 2^-23 of the weight goes on top of the rest, so that it is not zero either: a visible
// value of +-inf then meets two positive factors (0 inf and inf - inf are not numbers).  The rest
// is below 2^-7 of the weight and is rounded by at most 2^-8 of itself, together 2^-15, which the
// output's own rounding of 2^-8 covers.  (Below 2^-103 the rest leaves bf16's normal numbers.)
__device__ __forceinline__ void split_bf16(float e0, float e1, uint32_t& high, uint32_t& low) {
    constexpr float kOnTop = 1.f + 0x1p-23f;
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(high) : "f"(e1), "f"(e0));
    low = pack_bf16(fmaf(e0, kOnTop, -bf16lo(high)), fmaf(e1, kOnTop, -bf16hi(high)));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// The bits of x, or 0: a choice among registers (an index would move the array to memory).
__device__ __forceinline__ uint32_t bits_if(bool yes, float x) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tselp.b32 %0, %1, 0, p;\n\t}"
                 : "=r"(r)
                 : "r"(__float_as_uint(x)), "r"(yes ? 1u : 0u));
    return r;
}
// 16 bytes to shared memory, or 16 zero bytes; wait until at most n groups are outstanding.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async16_at(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

template <bool kFp8, int DT>
struct MmaShape {
    static constexpr int kThreads = 128, kWarps = 4;
    static constexpr int M = 16;
    static constexpr int KS = kFp8 ? 32 : 16;               // keys of a warp's step
    static constexpr int KT = KS * kWarps;                  // keys of a unit
    static constexpr int kRow = kFp8 ? DT : 2 * DT;         // bytes of a stored row
    static constexpr int kStage = 2 * KS * kRow;            // keys, then values
    static constexpr int kStages = DT <= 64 ? 4 : DT <= 128 ? 2 : 3;
    static constexpr int kWarpBytes = kStage * kStages;     // also holds a warp's result at the end
    static constexpr int kLd = DT + 8;                      // row of that result, floats
    static constexpr int kQBytes = M * DT * 2;
    static constexpr int kSmem = kWarps * kWarpBytes + kQBytes;
    static constexpr int kPerSm = kSmem > 113 * 1024 ? 1 : 3;
    static constexpr bool kQReg = DT <= 64;              // the queries' fragments stay in registers
    static_assert(M * kLd * 4 <= kWarpBytes, "a warp's result fits its ring");
};

// Byte offset of 16-byte chunk c of row r in rows of kRow bytes.
template <int kRow>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    if constexpr (kRow >= 128) return r * kRow + ((c ^ (r & 7)) << 4);
    else return r * kRow + ((c ^ ((r >> 1) & 3)) << 4);     // 64-byte rows: two rows share the 128 bytes of all banks
}

// Whether a 32-bit word holds a value that is not finite (8-bit: not a number), and the word
// with 0 in the place of each.
template <bool kFp8>
__device__ __forceinline__ bool any_odd(uint32_t u) {
    if constexpr (kFp8)
        return (u & 0x7Fu) == 0x7Fu || (u & 0x7F00u) == 0x7F00u || (u & 0x7F0000u) == 0x7F0000u || (u & 0x7F000000u) == 0x7F000000u;
    else
        return (u & 0x7F80u) == 0x7F80u || (u & 0x7F800000u) == 0x7F800000u;
}
template <bool kFp8>
__device__ __forceinline__ uint32_t without_odd(uint32_t u) {
    constexpr uint32_t kStep = kFp8 ? 8 : 16, kAll = kFp8 ? 0x7Fu : 0x7F80u, kField = kFp8 ? 0xFFu : 0xFFFFu;
#pragma unroll
    for (uint32_t i = 0; i < 32; i += kStep)
        if (((u >> i) & kAll) == kAll) u &= ~(kField << i);
    return u;
}

template <bool kFp8, int DT>
__global__ void __launch_bounds__(128, (MmaShape<kFp8, DT>::kPerSm)) attend_mma(const __grid_constant__ Args p) {
    using Sh = MmaShape<kFp8, DT>;
    constexpr int M = Sh::M, KS = Sh::KS, KT = Sh::KT, kRow = Sh::kRow, kStages = Sh::kStages;
    constexpr int kThreads = Sh::kThreads, kWarps = Sh::kWarps;
    constexpr int kSub = KS / 16;                            // 16-key blocks of a step
    constexpr int kChunks = kRow / 16;                       // 16-byte chunks of a stored row
    constexpr float kShift = kFp8 ? 14.f : 0.f;              // P carries 2^kShift
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long scratch[38];
    __shared__ float s_m[kWarps][M], s_l[kWarps][M], s_qs[M];
    __shared__ float2 s_row[M];
    __shared__ int s_flag;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, t = lane & 3;
    const float ninf = -__uint_as_float(0x7f800000u);
    unsigned char* ring = smem + w * Sh::kWarpBytes;
    const uint32_t ring_a = smem_u32(ring);
    unsigned char* s_q = smem + kWarps * Sh::kWarpBytes;
    const uint32_t q_a = smem_u32(s_q);
    const int esize = kFp8 ? 1 : 2;
    const int real_chunks = p.D * esize / 16;
    const bool whole_pages = p.page % 16 == 0;               // 16 keys (a step's or half of it) lie on one page
    const bool adjacent = whole_pages && p.D == DT;          // and fill the stored rows

    const Start st = find_start<M, KT, kThreads>(p, scratch);
    Walk<M, KT> walk(p, st);
    Piece pc;
    while (walk.next(pc)) {
        const int left = pc.r.n * p.G - pc.tile * M;
        const int valid = left < M ? left : M;
        // ---- the first keys and values are on their way before anything else
        const int steps = pc.u1 - pc.u0;
        const int key0 = pc.span.lo + pc.u0 * KT + w * KS;   // this warp's first key; then every KT
        // Where the keys of step s lie: the row (of D elements) of lane's key, or of the first of
        // its 16 where a page holds them.
        auto find_rows = [&](int s) -> int64_t {
            const int key = key0 + s * KT + (whole_pages ? lane & (KS - 16) : lane);
            if (s >= steps || key + (whole_pages ? 15 : 0) < pc.span.seen || key >= pc.span.hi || (!whole_pages && lane >= KS)) return 0;
            const int blk = key / p.page;
            return (static_cast<int64_t>(page_id(p, pc.b, blk)) * p.Hkv + pc.h) * p.page + (key - blk * p.page);
        };
        auto load = [&](int s, int64_t rows) {
            const int first = key0 + s * KT;
            if (s < steps && first < pc.span.hi && first + KS > pc.span.seen) {
                const uint32_t to = ring_a + (s % kStages) * Sh::kStage;
                const char* kc = static_cast<const char*>(p.kc);
                const char* vc = static_cast<const char*>(p.vc);
                int64_t run[kSub];                           // the first rows of the step's sixteens
#pragma unroll
                for (int b = 0; b < kSub; ++b) run[b] = kSub == 1 ? rows : __shfl_sync(0xffffffffu, rows, 16 * b);
                if (adjacent && first >= pc.span.seen && first + KS <= pc.span.hi) {
                    // sixteen rows are one run of bytes: 16 a lane, 512 on each time
                    constexpr int kIn = 16 * kChunks / 32;
#pragma unroll
                    for (int b = 0; b < kSub; ++b) {
                        const int64_t at = run[b] * kRow + lane * 16;
#pragma unroll
                        for (int i = 0; i < kIn; ++i) {
                            const int e = lane + 32 * (kIn * b + i);
                            const uint32_t d = to + chunk_at<kRow>(e / kChunks, e % kChunks);
                            cp_async16_at(d, kc + at + 512 * i);
                            cp_async16_at(d + KS * kRow, vc + at + 512 * i);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < KS * kChunks / 32; ++i) {
                        const int e = lane + 32 * i, r = e / kChunks, c = e % kChunks;
                        const int64_t mine = __shfl_sync(0xffffffffu, rows, whole_pages ? r & (KS - 16) : r);
                        const int64_t row = whole_pages ? mine + (r & 15) : mine;
                        const bool real = first + r >= pc.span.seen && first + r < pc.span.hi && c < real_chunks;
                        const int64_t at = real ? row * (p.D * esize) + c * 16 : 0;
                        const uint32_t d = to + chunk_at<kRow>(r, c);
                        copy16(d, kc + at, real);
                        copy16(d + KS * kRow, vc + at, real);
                    }
                }
            }
            copy_commit();
        };
        // The queries first (16-bit, swizzled, rows past the last zero): they arrive with the first keys.
        for (int e = tid; e < M * (DT / 8); e += kThreads) {
            const int m = e / (DT / 8), c = e - m * (DT / 8), qi = pc.tile * M + m;
            const bool real = m < valid && c * 8 < p.D;
            const int64_t at = real ? (static_cast<int64_t>(pc.r.row0) + qi / p.G) * p.q_stride +
                                          static_cast<int64_t>(pc.h * p.G + qi % p.G) * p.D + c * 8
                                    : 0;
            copy16(q_a + chunk_at<2 * DT>(m, c), static_cast<const __nv_bfloat16*>(p.q) + at, real);
        }
        int64_t ahead[kStages];
#pragma unroll
        for (int s = 0; s < kStages; ++s) ahead[s] = find_rows(s);
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) load(s, ahead[s]);
        int64_t rows = ahead[kStages - 1];
        copy_wait<kStages - 2>();
        __syncthreads();
        if (p.scale_log2 < 0.f) {                            // a negative scale's sign is the queries'
            for (int e = tid; e < M * DT / 2; e += kThreads) reinterpret_cast<uint32_t*>(s_q)[e] ^= 0x80008000u;
            __syncthreads();
        }
        if constexpr (kFp8) {
            // rows to f16: the largest element comes to 2^10 .. 2^11, and the columns of every
            // 16 into the order in which ldmatrix hands out the keys' bytes
            for (int m = w; m < M; m += kWarps) {
                float big = 0.f;
                for (int i = lane; i < DT / 2; i += 32) {
                    const uint32_t u = *reinterpret_cast<const uint32_t*>(s_q + chunk_at<2 * DT>(m, i >> 2) + (i & 3) * 4);
                    big = fmaxf(big, fmaxf(fabsf(bf16lo(u)), fabsf(bf16hi(u))));
                }
                big = warp_max(big);
                // 2^up and 2^-up by their exponent bits (up stays where both are normal numbers)
                int up = 0;
                if (big > 0.f && big < __uint_as_float(0x7f800000u)) up = min(10 - (static_cast<int>(__float_as_uint(big) >> 23) - 127), 126);
                const float grow = __uint_as_float(static_cast<uint32_t>(127 + up) << 23), back = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
                uint32_t own[DT / 64 > 0 ? (DT + 63) / 64 : 1];
#pragma unroll
                for (int k = 0; k < (DT + 63) / 64; ++k) {
                    const int i = lane + 32 * k;             // pair i: columns 2i, 2i + 1
                    const uint32_t u = i < DT / 2 ? *reinterpret_cast<const uint32_t*>(s_q + chunk_at<2 * DT>(m, i >> 2) + (i & 3) * 4) : 0u;
                    own[k] = pack_f16(bf16lo(u) * grow, bf16hi(u) * grow);
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < (DT + 63) / 64; ++k) {
                    const int i = lane + 32 * k;
                    // pair j of a block of 16 columns: 2t goes to pair t, 2t + 1 to pair 4 + t
                    const int j = i & 7, to = (i & ~7) + (j >> 1) + (j & 1) * 4;
                    if (i < DT / 2)
                        *reinterpret_cast<uint32_t*>(s_q + chunk_at<2 * DT>(m, to >> 2) + (to & 3) * 4) = own[k];
                }
                if (lane == 0) s_qs[m] = fabsf(p.scale_log2) * p.k_scale[pc.h] * back;
            }
            __syncthreads();
        }
        uint32_t qf[Sh::kQReg ? DT / 16 : 1][4];
        auto load_q = [&](int ks, uint32_t* a) {
            ldsm4(a, q_a + chunk_at<2 * DT>(lane & 15, 2 * ks + (lane >> 4)));
        };
        if constexpr (Sh::kQReg) {
#pragma unroll
            for (int ks = 0; ks < DT / 16; ++ks) load_q(ks, qf[ks]);
        }
        float sc[2], mx[2], l[2];
        float o[DT / 8][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            sc[r] = fmaxf(kFp8 ? s_qs[g + 8 * r] : fabsf(p.scale_log2), 1.17549435e-38f);   // -inf times it is -inf
            mx[r] = ninf;
            l[r] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < DT / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.f;

        const int pos_lo = pc.r.len + pc.tile * M / p.G, pos_hi = pc.span.hi - 1;   // the tile's first and last position
        for (int s = 0; s < steps; ++s) {
            copy_wait<kStages - 2>();
            __syncwarp();
            load(s + kStages - 1, rows);
            rows = find_rows(s + kStages);
            const int first = key0 + s * KT;
            if (first >= pc.span.hi || first + KS <= pc.span.seen) continue;
            const uint32_t k_a = ring_a + (s % kStages) * Sh::kStage, v_a = k_a + KS * kRow;

            // ---- S = Q K^T
            float sv[2 * kSub][4];
#pragma unroll
            for (int n = 0; n < 2 * kSub; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) sv[n][i] = 0.f;
#pragma unroll
            for (int ks = 0; ks < DT / 16; ++ks) {
                uint32_t kf[4];
                if constexpr (kFp8) ldsm4(kf, k_a + chunk_at<kRow>(lane, ks));
                else ldsm4(kf, k_a + chunk_at<kRow>((lane & 7) + (lane >> 4) * 8, 2 * ks + ((lane >> 3) & 1)));
                uint32_t qa[4];
                const uint32_t* a = qa;
                if constexpr (Sh::kQReg) a = qf[ks];
                else load_q(ks, qa);
                if constexpr (kFp8) {
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        mma16816<true>(sv[n], a, e4m3x2_f16x2(kf[n]), e4m3x2_f16x2(kf[n] >> 16));
                } else {
                    mma16816<false>(sv[0], a, kf[0], kf[1]);
                    mma16816<false>(sv[1], a, kf[2], kf[3]);
                }
            }
            // ---- scores; hidden keys at -inf.  Their scale (to units of log 2) is not negative, so the
            // largest is found before scaling and the scaling is part of the exponent's addition.
            const bool masked = first + KS - 1 > pos_lo || (p.window > 0 && first <= pos_hi - p.window);
            uint32_t hidden[2];                          // bit 2n + i: key 8n + 2t + i is hidden from row g (+ 8)
            float nm[2];
            bool moved = false;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                hidden[r] = 0;
                if (masked) {
                    const int pos = pc.r.len + (pc.tile * M + g + 8 * r) / p.G;
#pragma unroll
                    for (int n = 0; n < 2 * kSub; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int key = first + 8 * n + 2 * t + i;
                            if (key > pos || key >= pc.span.hi || (p.window > 0 && key <= pos - p.window)) {
                                hidden[r] |= 1u << (2 * n + i);
                                sv[n][2 * r + i] = ninf;
                            }
                        }
                }
                float m2[2] = {ninf, ninf};
#pragma unroll
                for (int n = 0; n < 2 * kSub; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) m2[i] = fmaxf(m2[i], sv[n][2 * r + i]);
                float mm = fmaxf(m2[0], m2[1]);
                mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, 1));
                mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, 2));
                mm = fmaxf(mx[r], mm == ninf ? ninf : mm * sc[r]);
                nm[r] = mm;
                moved |= mm != mx[r];
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float a = fast_exp2(mx[r] - (nm[r] == ninf ? 0.f : nm[r]));
                    l[r] *= a;
                    mx[r] = nm[r];
#pragma unroll
                    for (int n = 0; n < DT / 8; ++n) {
                        o[n][2 * r] *= a;
                        o[n][2 * r + 1] *= a;
                    }
                }
            }
            // ---- P
            uint32_t ph[kSub][4], pl[kSub][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float use = (mx[r] == ninf ? 0.f : mx[r]) - kShift;
#pragma unroll
                for (int n = 0; n < 2 * kSub; ++n) {
                    const float e0 = fast_exp2(fmaf(sv[n][2 * r], sc[r], -use));
                    const float e1 = fast_exp2(fmaf(sv[n][2 * r + 1], sc[r], -use));
                    l[r] += e0 + e1;
                    sv[n][2 * r] = e0;
                    sv[n][2 * r + 1] = e1;
                    const int at = (n & 1) * 2 + r;
                    if constexpr (kFp8) {
                        ph[n >> 1][at] = pack_f16(e0, e1);
                    } else {
                        split_bf16(e0, e1, ph[n >> 1][at], pl[n >> 1][at]);
                    }
                }
            }
            // ---- O += P V.  A hidden key's P is 0, which keeps its value out as long as that is
            // finite.  Steps with hidden keys look: values that are not finite are added here, to
            // the rows that see them, and become 0 for the product.
            if (masked) {
                unsigned char* vb = ring + (s % kStages) * Sh::kStage + KS * kRow;
                bool odd = false;
                for (int i = lane; i < KS * kRow / 4; i += 32) odd |= any_odd<kFp8>(reinterpret_cast<const uint32_t*>(vb)[i]);
                if (__any_sync(0xffffffffu, odd)) {
                    for (int j = 0; j < KS; ++j) {
                        const int src = g * 4 + ((j & 7) >> 1);
                        float e[2];
                        bool in[2];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            uint32_t mine = 0;
#pragma unroll
                            for (int k = 0; k < 4 * kSub; ++k) mine |= bits_if(k == 2 * (j >> 3) + (j & 1), sv[k >> 1][2 * r + (k & 1)]);
                            e[r] = __uint_as_float(__shfl_sync(0xffffffffu, mine, src));
                            in[r] = !(__shfl_sync(0xffffffffu, hidden[r], src) >> (2 * (j >> 3) + (j & 1)) & 1u);
                        }
#pragma unroll
                        for (int n = 0; n < DT / 8; ++n) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                // column of accumulator i of tile n, as the products below leave it
                                const int d = kFp8 ? (n >> 1) * 16 + 4 * t + 2 * i + (n & 1) : n * 8 + 2 * t + i;
                                const unsigned char* at = vb + chunk_at<kRow>(j, d * esize / 16) + d * esize % 16;
                                const uint32_t bits = kFp8 ? *at : *reinterpret_cast<const uint16_t*>(at);
                                if (any_odd<kFp8>(bits)) {
                                    const float v = kFp8 ? __uint_as_float(0x7fffffffu) : bf16lo(bits);
                                    if (in[0]) o[n][i] = fmaf(e[0], v, o[n][i]);
                                    if (in[1]) o[n][2 + i] = fmaf(e[1], v, o[n][2 + i]);
                                }
                            }
                        }
                    }
                    __syncwarp();
                    for (int i = lane; i < KS * kRow / 4; i += 32) {
                        uint32_t& u = reinterpret_cast<uint32_t*>(vb)[i];
                        u = without_odd<kFp8>(u);
                    }
                    __syncwarp();
                }
            }
            if constexpr (kFp8) {
#pragma unroll
                for (int c = 0; c < DT / 16; ++c) {
                    uint32_t vf[4];
                    ldsm4_t(vf, v_a + chunk_at<kRow>(lane, c));
                    uint32_t ev[4], od[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t x = __byte_perm(vf[i], 0, 0x3120);      // even columns' two keys, then the odd ones'
                        ev[i] = e4m3x2_f16x2(x);
                        od[i] = e4m3x2_f16x2(x >> 16);
                    }
#pragma unroll
                    for (int b = 0; b < kSub; ++b) {
                        mma16816<true>(o[2 * c], ph[b], ev[2 * b], ev[2 * b + 1]);
                        mma16816<true>(o[2 * c + 1], ph[b], od[2 * b], od[2 * b + 1]);
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < DT / 8; c += 2) {
                    uint32_t vf[4];
                    ldsm4_t(vf, v_a + chunk_at<kRow>(lane & 15, c + (lane >> 4)));
                    mma16816<false>(o[c], ph[0], vf[0], vf[1]);
                    mma16816<false>(o[c + 1], ph[0], vf[2], vf[3]);
                    mma16816<false>(o[c], pl[0], vf[0], vf[1]);
                    mma16816<false>(o[c + 1], pl[0], vf[2], vf[3]);
                }
            }
        }
        copy_wait<0>();
        __syncwarp();

        // ---- the four warps' results join
        float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float sum = l[r];
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            const int m = g + 8 * r;
            if (t == 0) {
                s_m[w][m] = mx[r];
                s_l[w][m] = sum;
            }
#pragma unroll
            for (int n = 0; n < DT / 8; ++n) {
                if constexpr (kFp8) {
                    if ((n & 1) == 0)
                        *reinterpret_cast<float4*>(mine + m * Sh::kLd + n * 8 + 4 * t) =
                            make_float4(o[n][2 * r], o[n + 1][2 * r], o[n][2 * r + 1], o[n + 1][2 * r + 1]);
                } else {
                    *reinterpret_cast<float2*>(mine + m * Sh::kLd + n * 8 + 2 * t) =
                        make_float2(o[n][2 * r], o[n][2 * r + 1]);
                }
            }
        }
        __syncthreads();
        const bool whole = pc.whole();
        if (tid < M) {
            // a row's maximum and sum, and each warp's factor in its output (the values' scale and, where
            // this is the whole, the sum with it)
            float big = ninf, sum = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) big = fmaxf(big, s_m[i][tid]);
            const float use = big == ninf ? 0.f : big, vs = kFp8 ? p.v_scale[pc.h] : 1.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) sum += s_l[i][tid] * fast_exp2(s_m[i][tid] - use);
            const float f = !whole ? vs : sum != 0.f ? vs / sum : 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) s_m[i][tid] = f * fast_exp2(s_m[i][tid] - use);
            if (tid < valid) {
                if (!whole) {
                    reinterpret_cast<float2*>(p.part_ml)[part_place(blockIdx.x, pc.u0 == 0) * M + tid] = make_float2(big - kShift, sum);
                } else if (p.lse != nullptr) {
                    const int qi = pc.tile * M + tid;
                    p.lse[(static_cast<int64_t>(pc.r.row0) + qi / p.G) * p.Hq + pc.h * p.G + qi % p.G] = lse_of(big - kShift, sum);
                }
            }
        }
        __syncthreads();
        const int four = p.D / 4;
        float* part = p.part_o + part_place(blockIdx.x, pc.u0 == 0) * M * p.D;
#pragma unroll 2
        for (int e = tid; e < valid * four; e += kThreads) {
            const int m = e / four, d = (e - m * four) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float f = s_m[i][m];
                const float4 v = *reinterpret_cast<const float4*>(smem + i * Sh::kWarpBytes + (m * Sh::kLd + d) * 4);
                x.x = fmaf(v.x, f, x.x);
                x.y = fmaf(v.y, f, x.y);
                x.z = fmaf(v.z, f, x.z);
                x.w = fmaf(v.w, f, x.w);
            }
            if (whole) {
                const int qi = pc.tile * M + m, head = pc.h * p.G + qi % p.G;
                const int64_t row = static_cast<int64_t>(pc.r.row0) + qi / p.G;
                store_four(static_cast<__nv_bfloat16*>(p.out) + (row * p.Hq + head) * p.D + d, x);
            } else {
                store_four(part + m * p.D + d, x);
            }
        }
        if (!whole && part_done(p, pc, st, &s_flag, tid, [] { __syncthreads(); })) 
            join_parts<__nv_bfloat16, M, kThreads>(p, pc, st, s_row, tid, [] { __syncthreads(); });
        __syncthreads();
    }
    if (blockIdx.x == 0) head_cleared();
}

template <bool kFp8, int DT>
dspark_status_t launch_mma(const Args& p, cudaStream_t s) {
    using Sh = MmaShape<kFp8, DT>;
    static OncePerDevice once;
    const int dev = current_device();
    if (once.run(dev, [] {
            return cudaFuncSetAttribute(attend_mma<kFp8, DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
        }) != cudaSuccess)
        return DSPARK_ERR_CUDA;
    const int grid = grid_for(sm_count(dev) * Sh::kPerSm, Sh::M);
    if (grid < 1) return DSPARK_ERR_CUDA;
    return launch_cleared(p.status, kHeadBytes, attend_mma<kFp8, DT>, dim3(grid), Sh::kThreads, Sh::kSmem, s, p);
}

}  // namespace attn
}  // namespace dspark
