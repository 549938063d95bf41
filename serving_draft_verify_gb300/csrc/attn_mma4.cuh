// Attention over a 4-bit cache (kv_store.cuh has the format): 8, 16, 24 or 32 query rows of a key head
// at a time on the warp-level tensor instructions.
//
// The work is divided as in attn_mma.cuh: each of a block's four warps takes 32 keys of every unit of
// 128, with a ring of its own, its own running maximum and sum and its own part of the output.  Turning codes into
// operands is what most instructions do (a conversion for two elements and a multiplication for two, 256 of a
// warp's 650 for 32 keys of 128 elements and 8 query rows), so keys and values
// are the side of the products that has 16 rows and the queries the one that has 8: a step for up to 8 query rows (plain
// decoding with groups of 8 and fewer) then costs half the products and half the exponentials.  No pipe is full, though: what
// it waits for most is the fixed latency between dependent instructions, with two or three warps a scheduler.
//
// 32 heads on 8 of 128, pages of 16: 64 requests of one row and up to 16384 keys 147 us for 676 MB (4.6 TB/s; three blocks an
// SM; with a quarter of the requests issuing in 50 % of the cycles, ALU pipe 41 %, tensor pipe 28 %); 16 requests of 8 rows and
// up to 32768 keys 203 us (32 rows a tile, two blocks an SM by 255 registers, 72 bytes of spill stores and 104 of loads that
// are a thousandth of the instructions; issuing in 48 %, tensor pipe 41 %); 128 requests of
// up to 17 rows and 6000 keys 380 us (three tiles of 24).  Keys as the side of 8 took 235, 257 and 500; on
// tcgen05, codes converted into shared memory by the way, 400, 271 and 640.
//
//   S' = K Q'    m16n8k16 in f16, query rows as columns,
//   P' = 2^((S' - m) c + 14), rounded to 11 bits; the sum carries the factor 2^14 too,
//   O' += V' P'  P' turned from accumulators to operands by movmatrix.
//
// m is the largest product of a row so far, before its scale c (to units of log 2), or one whose score is up to 1 below
// the largest: f16 has room for that, so the maximum has to be found across the warp, and the output scaled, only in steps
// where a vote says so.  The difference is taken before it is scaled: m c rounded to float32 is off by 2 and more
// from 2^25 on, which took P' past f16's largest.
//
// A stored value is code x block scale x head scale.  The product of the first two is exact in f16; the
// head's scale goes into the scores' scale (keys) and the end result (values).  Q's rows are scaled by a
// power of two into f16's range.
//
// Codes as operands.  ldmatrix hands a thread 4 adjacent bytes of one key, elements 8t .. 8t + 7 of 32:
// two steps of the first product take them as they come (k = 2t, 2t + 1, 2t + 8, 2t + 9 stand for elements
// 8t .. 8t + 3, then 8t + 4 .. 8t + 7), and Q's elements are those 16 bytes of its row, no permutation
// needed.  All four bytes lie in one block of 16: one scale.  For the second product the transposing ldmatrix hands out
// two bytes (elements 4g .. 4g + 3) of key 2t and the same two of key 2t + 1, whose conversions hold two elements of a key
// where the operand wants an element of two keys.  For 8 query rows they are taken as they are, as if an
// element's two neighbours were two keys: once with weights (P, 0), which gives the even elements, once with (0, P) for the
// odd ones.  That is twice the products, which are few.  For more rows the halves are paired: a multiplication by
// (0, s') and one by (s, 0) that adds to it do that and the scaling at once, on the pipe that has less to do than
// the one that converts and permutes.  Either way rows g and g + 8 of tile r are elements 4g + r and 4g + 2 + r, and a
// thread ends with four adjacent elements of its rows.
#pragma once

#include <cuda_fp16.h>

#include "attn_mma.cuh"

namespace dspark {
namespace attn {

template <int DT, int NT>
struct Mma4Shape {
    static constexpr int kThreads = 128, kWarps = 4;
    static constexpr int M = 8 * NT;                        // query rows of a tile
    static constexpr int KS = 32;                           // keys of a warp's step
    static constexpr int KT = KS * kWarps;                  // keys of a unit
    // What a piece costs by itself, in units (12,200 cycles and 3,900 with 32 query rows, 6,000 and 2,200 with 8, by the
    // SM's clock before the results were written by columns).  256 requests of up to 500 keys: 8 rows 109 us, without
    // 135, with five 114; 1 row 48, 60 and 48; a prompt of 2048 rows 264, 347 and 277.
    static constexpr int kOver = 3;
    static constexpr int kRow = DT / 2;                     // bytes of a row's codes
    static constexpr int kScale = DT / 16;                  // and of its scales
    static constexpr int kStage = 2 * KS * (kRow + kScale); // codes of keys, of values, scales of keys, of values
    // Blocks an SM, by registers.  Four of 8 rows and heads of 128 have room for two stages only: 154 us for 150
    // (heads of 64 105, with three blocks 109); two blocks 156.
    static constexpr int kPerSm = NT >= 3 || DT > 128 ? 2 : NT == 1 && DT <= 64 ? 4 : 3;
    static constexpr int kStages = DT <= 64 ? 4 : DT <= 128 ? (NT == 4 ? 4 : 3) : 2;
    static constexpr int kWarpBytes = kStage * kStages;     // also holds a warp's result at the end
    static constexpr int kLd = DT + 4;                      // row of that result, floats
    static constexpr int kQBytes = M * DT * 2;
    static constexpr int kSmem = kWarps * kWarpBytes + kQBytes;
    static constexpr bool kQReg = NT * DT <= 128;           // the queries' operands stay in registers
    static_assert(M * kLd * 4 <= kWarpBytes, "a warp's result fits its ring");
    static_assert(kPerSm * (kSmem + 3072) <= 227 * 1024, "shared memory");
};

// Byte offset of 16-byte chunk c of row r in rows of kRow bytes, free of conflicts for eight rows.
template <int kRow>
__device__ __forceinline__ uint32_t code_at(int r, int c) {
    if constexpr (kRow >= 64) return chunk_at<kRow>(r, c);
    else return r * kRow + ((c ^ ((r >> 2) & 1)) << 4);
}
// Byte offset of 16-byte chunk c of query row m: a quarter warp reads four chunks of two rows.
template <int DT>
__device__ __forceinline__ uint32_t query_at(int m, int c) {
    return m * (2 * DT) + ((c ^ ((m & 1) << 2)) << 4);
}
// 4 bytes to shared memory, the first n of them read, the others zero.
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// The low (0) or the high (1) half twice (as an operand this costs nothing, which a byte permutation
// does); in the low half, over 0; in the high half, over 0.
__device__ __forceinline__ uint32_t both(uint32_t x, int high) {
    uint32_t r;
    if (high) asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(r) : "r"(x));
    else asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t in_low(uint32_t x, int high) { return high ? x >> 16 : x & 0xFFFFu; }
__device__ __forceinline__ uint32_t in_high(uint32_t x, int high) { return high ? x & 0xFFFF0000u : x << 16; }
// An 8 x 8 matrix of f16, two adjacent elements of a row a thread, transposed.
__device__ __forceinline__ uint32_t turned8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Of a row's DT / 16 scale bytes (kWords words), every second one from `odd` on: one f16 for each 32
// elements, two to a word.
template <int DT>
__device__ __forceinline__ void half_scales(const uint32_t* w, uint32_t pick, uint32_t* out) {
    if constexpr (DT == 64) {
        out[0] = e4m3x2_f16x2(__byte_perm(w[0], 0, pick));
    } else {
#pragma unroll
        for (int i = 0; i < DT / 128; ++i) e4m3x4_f16(__byte_perm(w[2 * i], w[2 * i + 1], pick), out[2 * i], out[2 * i + 1]);
    }
}
template <int kWords>
__device__ __forceinline__ void load_words(const unsigned char* at, uint32_t* w) {
    if constexpr (kWords == 1) {
        w[0] = *reinterpret_cast<const uint32_t*>(at);
    } else if constexpr (kWords == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(at);
        w[0] = x.x, w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 x = *reinterpret_cast<const uint4*>(at + 16 * i);
            w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
        }
    }
}

template <int DT, int NT>
__global__ void __launch_bounds__(128, (Mma4Shape<DT, NT>::kPerSm)) attend_mma4(const __grid_constant__ Args p) {
    using Sh = Mma4Shape<DT, NT>;
    constexpr int M = Sh::M, KS = Sh::KS, KT = Sh::KT, kRow = Sh::kRow, kScale = Sh::kScale, kStages = Sh::kStages;
    constexpr int kThreads = Sh::kThreads, kWarps = Sh::kWarps;
    constexpr int kChunks = kRow / 16;                       // 16-byte chunks of a row's codes
    constexpr int kV = KS * kRow, kKs = 2 * KS * kRow, kVs = kKs + KS * kScale;      // parts of a stage behind the keys
    constexpr int kPairs = (DT + 63) / 64;                   // words of scales a thread keeps of one row
    constexpr float kShift = 14.f;                           // P carries 2^kShift
    constexpr float kNone = -3.40282347e38f;                 // below any sum of products, and finite
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
    const int real_chunks = p.D / 32;
    const bool whole_pages = p.page % 16 == 0;               // 16 keys (half of a step's) lie on one page
    const bool adjacent = whole_pages && p.D == DT;          // and fill the rows
    const uint32_t k_pick = t < 2 ? 0x6420 : 0x7531, v_pick = g < 4 ? 0x6420 : 0x7531;
    const uint32_t place0 = code_at<kRow>(lane / kChunks, lane % kChunks);
    const char* kc = static_cast<const char*>(p.kc);
    const char* vc = static_cast<const char*>(p.vc);

    const Start st = find_start<M, KT, kThreads, Sh::kOver>(p, scratch);
    Walk<M, KT, Sh::kOver> walk(p, st);
    Piece pc;
    while (walk.next(pc)) {
        const int left = pc.r.n * p.G - pc.tile * M;
        const int valid = left < M ? left : M;
        // ---- the first keys and values are on their way before anything else
        const int steps = pc.u1 - pc.u0;
        const int key0 = pc.span.lo + pc.u0 * KT + w * KS;   // this warp's first key; then every KT
        // Where the keys of step s lie: the page's id and the row in it of lane's key, or of the first of
        // its 16 where a page holds them.  The id is looked at only when the copies are issued, a step later:
        // checking it here would wait for it.
        struct Place {
            int id, row;
        };
        const int32_t* table = p.table + static_cast<int64_t>(pc.b) * p.ld_table;
        auto find_rows = [&](int s) -> Place {
            const int key = key0 + s * KT + (whole_pages ? lane & 16 : lane);
            if (s >= steps || key + (whole_pages ? 15 : 0) < pc.span.seen || key >= pc.span.hi) return Place{0, 0};
            const int blk = p.page_shift >= 0 ? key >> p.page_shift : key / p.page;
            return Place{__ldg(table + blk), key - blk * p.page};
        };
        auto load = [&](int s, uint32_t to, const Place& at) {
            const int first = key0 + s * KT;
            if (s < steps && first < pc.span.hi && first + KS > pc.span.seen) {
                const int64_t page = (static_cast<int64_t>(checked_page(p, at.id)) * p.Hkv + pc.h) * p.g4.whole;
                const int64_t code = page + at.row * p.g4.code, scale = page + (p.g4.codes + at.row * p.g4.scale);
                if (adjacent && first >= pc.span.seen && first + KS <= pc.span.hi) {
                    // sixteen rows are one run of codes and one of scales: 16 bytes a lane
                    constexpr int kIn = 16 * kChunks / 32;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int64_t run = __shfl_sync(0xffffffffu, code, 16 * b) + lane * 16;
#pragma unroll
                        for (int i = 0; i < kIn; ++i) {
                            const int e = lane + 32 * (kIn * b + i);
                            // 32 chunks of whole eights of rows on, the swizzle is the same
                            const uint32_t d = to + (32 / kChunks % 8 == 0 ? place0 + 512 * (kIn * b + i) : code_at<kRow>(e / kChunks, e % kChunks));
                            cp_async16_at(d, kc + run + 512 * i);
                            cp_async16_at(d + kV, vc + run + 512 * i);
                        }
                    }
                    if (lane % 16 < kScale) {
                        cp_async16_at(to + kKs + (lane / 16 * kScale + lane % 16) * 16, kc + scale + lane % 16 * 16);
                        cp_async16_at(to + kVs + (lane / 16 * kScale + lane % 16) * 16, vc + scale + lane % 16 * 16);
                    }
                } else {
                    const int in16 = whole_pages ? lane & 15 : 0;            // of lane's key in its 16
#pragma unroll
                    for (int i = 0; i < KS * kChunks / 32; ++i) {
                        const int e = lane + 32 * i, r = e / kChunks, c = e % kChunks;
                        const int64_t run = __shfl_sync(0xffffffffu, code, r) + (whole_pages ? (r & 15) * p.g4.code : 0);
                        const bool real = first + r >= pc.span.seen && first + r < pc.span.hi && c < real_chunks;
                        const int64_t from = real ? run + c * 16 : 0;
                        const uint32_t d = to + code_at<kRow>(r, c);
                        copy16(d, kc + from, real);
                        copy16(d + kV, vc + from, real);
                    }
                    const bool real = first + lane >= pc.span.seen && first + lane < pc.span.hi;
                    const int64_t from = real ? scale + in16 * p.g4.scale : 0;
#pragma unroll
                    for (int i = 0; i < kScale / 4; ++i) {
                        const int n = real ? min(4, max(0, p.D / 16 - 4 * i)) : 0;
                        copy4(to + kKs + lane * kScale + 4 * i, kc + from + (n > 0 ? 4 * i : 0), n);
                        copy4(to + kVs + lane * kScale + 4 * i, vc + from + (n > 0 ? 4 * i : 0), n);
                    }
                }
            }
            copy_commit();
        };
        Place ahead[kStages];
#pragma unroll
        for (int s = 0; s < kStages; ++s) ahead[s] = find_rows(s);
        const float ks = fabsf(p.scale_log2) * p.k_scale[pc.h];
        // The queries first (16-bit, rows past the last zero): they arrive with the first keys.
        for (int e = tid; e < M * (DT / 8); e += kThreads) {
            const int m = e / (DT / 8), c = e - m * (DT / 8), qi = pc.tile * M + m;
            const bool real = m < valid && c * 8 < p.D;
            const int64_t at = real ? (static_cast<int64_t>(pc.r.row0) + qi / p.G) * p.q_stride +
                                          static_cast<int64_t>(pc.h * p.G + qi % p.G) * p.D + c * 8
                                    : 0;
            copy16(q_a + query_at<DT>(m, c), static_cast<const __nv_bfloat16*>(p.q) + at, real);
        }
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) load(s, ring_a + s * Sh::kStage, ahead[s]);
        Place rows = ahead[kStages - 1];
        copy_wait<kStages - 2>();
        __syncthreads();
        // Rows to f16, in place, eight a warp and four lanes a row: the largest element comes to 2^10 .. 2^11, a
        // negative scale's sign with it.
        if (w < NT) {
            const int m = 8 * w + g;
            uint4 own[DT / 32];
            float big = 0.f;
#pragma unroll
            for (int c = 0; c < DT / 32; ++c) {
                own[c] = *reinterpret_cast<const uint4*>(s_q + query_at<DT>(m, 4 * c + t));
                const uint32_t u[4] = {own[c].x, own[c].y, own[c].z, own[c].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) big = fmaxf(big, fmaxf(fabsf(bf16lo(u[i])), fabsf(bf16hi(u[i]))));
            }
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            // 2^up and 2^-up by their exponent bits (up stays where both are normal numbers)
            int up = 0;
            if (big > 0.f && big < __uint_as_float(0x7f800000u)) up = min(10 - (static_cast<int>(__float_as_uint(big) >> 23) - 127), 126);
            const float grow = __uint_as_float((p.scale_log2 < 0.f ? 0x80000000u : 0u) | static_cast<uint32_t>(127 + up) << 23);
            auto f16 = [&](uint32_t u) { return pack_f16(bf16lo(u) * grow, bf16hi(u) * grow); };
#pragma unroll
            for (int c = 0; c < DT / 32; ++c)
                *reinterpret_cast<uint4*>(s_q + query_at<DT>(m, 4 * c + t)) = make_uint4(f16(own[c].x), f16(own[c].y), f16(own[c].z), f16(own[c].w));
            // not 0: -inf times it is -inf, and kNone times it is below -1
            if (t == 0) s_qs[m] = fmaxf(ks * __uint_as_float(static_cast<uint32_t>(127 - up) << 23), 1.17549435e-38f);
        }
        __syncthreads();
        uint4 qf[Sh::kQReg ? DT / 32 : 1][Sh::kQReg ? NT : 1];
        auto load_q = [&](int c, int n) { return *reinterpret_cast<const uint4*>(s_q + query_at<DT>(8 * n + g, 4 * c + t)); };
        if constexpr (Sh::kQReg) {
#pragma unroll
            for (int c = 0; c < DT / 32; ++c)
#pragma unroll
                for (int n = 0; n < NT; ++n) qf[c][n] = load_q(c, n);
        }
        // This thread's query rows: 8n + 2t and 8n + 2t + 1, shared with the seven other g.
        float sc[NT][2], mx[NT][2], l[NT][2];                // mx: m, kNone before a key is seen
        float o[NT][DT / 16][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                sc[n][r] = s_qs[8 * n + 2 * t + r];
                mx[n][r] = kNone;
                l[n][r] = 0.f;
            }
#pragma unroll
            for (int d = 0; d < DT / 16; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][d][i] = 0.f;
        }

        const int pos_lo = pc.r.len + pc.tile * M / p.G, pos_hi = pc.span.hi - 1;   // the tile's first and last position
        int now = 0, last = (kStages - 1) * Sh::kStage;      // the step's stage and the one before, in the ring
        for (int s = 0; s < steps; ++s) {
            copy_wait<kStages - 2>();
            __syncwarp();
            load(s + kStages - 1, ring_a + last, rows);
            rows = find_rows(s + kStages);
            const int first = key0 + s * KT;
            unsigned char* stage = ring + now;
            const uint32_t k_a = ring_a + now, v_a = k_a + kV;
            last = now;
            now = now == (kStages - 1) * Sh::kStage ? 0 : now + Sh::kStage;
            if (first >= pc.span.hi || first + KS <= pc.span.seen) continue;

            // ---- S' = K Q'
            uint32_t scale[4][kPairs];                       // of keys 8i + g: this thread's block of every 32 elements
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t x[kScale / 4];
                load_words<kScale / 4>(stage + kKs + (8 * i + g) * kScale, x);
                half_scales<DT>(x, k_pick, scale[i]);
            }
            float sv[NT][2][4];                              // keys 16b + g (+ 8 from the third on), rows 2t, 2t + 1
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sv[n][b][i] = 0.f;
#pragma unroll
            for (int c = 0; c < DT / 32; ++c) {
                uint32_t kf[4];
                ldsm4(kf, k_a + code_at<kRow>(lane, c));
                uint4 q[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if constexpr (Sh::kQReg) q[n] = qf[c][n];
                    else q[n] = load_q(c, n);
                }
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t h[2][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        e2m1x8_f16(kf[2 * b + i], h[i]);
                        const uint32_t a = both(scale[2 * b + i][c / 2], c & 1);
#pragma unroll
                        for (int j = 0; j < 4; ++j) h[i][j] = hmul2(h[i][j], a);
                    }
                    const uint32_t a0[4] = {h[0][0], h[1][0], h[0][1], h[1][1]}, a1[4] = {h[0][2], h[1][2], h[0][3], h[1][3]};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma16816<true>(sv[n][b], a0, q[n].x, q[n].y);
                        mma16816<true>(sv[n][b], a1, q[n].z, q[n].w);
                    }
                }
            }
            // ---- scores; hidden keys at -inf.  Their scale is positive, so the largest is found before scaling.
            const bool masked = first + KS - 1 > pos_lo || (p.window > 0 && first <= pos_hi - p.window);
            uint32_t hidden[NT];                             // bit 4r + i: key 8i + g is hidden from row 2t + r
            bool above = false;
            float big[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                hidden[n] = 0;
                if (masked) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int pos = pc.r.len + (pc.tile * M + 8 * n + 2 * t + r) / p.G;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = first + 8 * i + g;
                            if (key > pos || key >= pc.span.hi || (p.window > 0 && key <= pos - p.window)) {
                                hidden[n] |= 1u << (4 * r + i);
                                sv[n][i >> 1][(i & 1) * 2 + r] = ninf;
                            }
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    big[n][r] = fmaxf(fmaxf(sv[n][0][r], sv[n][0][2 + r]), fmaxf(sv[n][1][r], sv[n][1][2 + r]));
                    above |= (big[n][r] - mx[n][r]) * sc[n][r] > 1.f;
                }
            }
            if (__any_sync(0xffffffffu, above)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float m = big[n][r];
#pragma unroll
                        for (int x = 4; x < 32; x *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
                        m = fmaxf(mx[n][r], m);
                        const float a = fast_exp2((mx[n][r] - m) * sc[n][r]);
                        l[n][r] *= a;
                        mx[n][r] = m;
#pragma unroll
                        for (int d = 0; d < DT / 16; ++d) {
                            o[n][d][r] *= a;
                            o[n][d][2 + r] *= a;
                        }
                    }
            }
            // ---- P'
            uint32_t pb[NT][2][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float e0 = fast_exp2(fmaf(sv[n][b][2 * i] - mx[n][0], sc[n][0], kShift));
                        const float e1 = fast_exp2(fmaf(sv[n][b][2 * i + 1] - mx[n][1], sc[n][1], kShift));
                        l[n][0] += e0;
                        l[n][1] += e1;
                        pb[n][b][i] = turned8x8(pack_f16(e0, e1));
                    }
            }
            // ---- O' += V' P'.  A hidden key's P is 0, which keeps its value out as long as that is a number.
            // Steps with hidden keys look at the scales: a block that is not a number is added here, to
            // the rows that see it, and becomes 0 for the product.
            if (masked) {
                unsigned char* vs = stage + kVs;
                bool odd = false;
                for (int i = lane; i < KS * kScale / 4; i += 32) odd |= any_odd<true>(reinterpret_cast<const uint32_t*>(vs)[i]);
                if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
                    for (int j = 0; j < KS; ++j) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint32_t seen = ~__shfl_sync(0xffffffffu, hidden[n], (j & 7) * 4 + t) >> (j >> 3);
#pragma unroll
                            for (int c = 0; c < DT / 32; ++c)
                                if (any_odd<true>(vs[j * kScale + 2 * c + (g >> 2)])) {
#pragma unroll
                                    for (int r = 0; r < 2; ++r)
                                        if (seen >> (4 * r) & 1u)
                                            o[n][2 * c][r] = o[n][2 * c][2 + r] = o[n][2 * c + 1][r] = o[n][2 * c + 1][2 + r] = __uint_as_float(0x7fffffffu);
                                }
                        }
                    }
                    __syncwarp();
                    for (int i = lane; i < KS * kScale / 4; i += 32) {
                        uint32_t& u = reinterpret_cast<uint32_t*>(vs)[i];
                        u = without_odd<true>(u);
                    }
                    __syncwarp();
                }
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t vscale[2][2][kPairs];               // of keys 16b + 8i + 2t and the next
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t x[kScale / 2];
                    load_words<kScale / 2>(stage + kVs + (16 * b + 8 * i + 2 * t) * kScale, x);
                    half_scales<DT>(x, v_pick, vscale[i][0]);
                    half_scales<DT>(x + kScale / 4, v_pick, vscale[i][1]);
                }
#pragma unroll
                for (int c2 = 0; c2 < DT / 64; ++c2) {
                    uint32_t vf[4];                          // keys 16b .. and 16b + 8 .. of 32 elements, then of the next 32
                    ldsm4_t(vf, v_a + code_at<kRow>(16 * b + (lane & 15), 2 * c2 + (lane >> 4)));
#pragma unroll
                    for (int odd = 0; odd < 2; ++odd) {
                        if constexpr (NT == 1) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                uint32_t h[4];
                                e2m1x8_f16(vf[2 * odd + i], h);
                                const uint32_t s0 = both(vscale[i][0][c2], odd), s1 = both(vscale[i][1][c2], odd);
                                const uint32_t a[4] = {hmul2(h[0], s0), hmul2(h[1], s0), hmul2(h[2], s1), hmul2(h[3], s1)};
                                const uint32_t x = pb[0][b][i];
                                mma16816<true>(o[0][4 * c2 + 2 * odd], a, x & 0xFFFFu, x >> 16);
                                mma16816<true>(o[0][4 * c2 + 2 * odd + 1], a, x << 16, x & 0xFFFF0000u);
                            }
                        } else {
                            uint32_t a[2][4];                // of tile j: rows g and g + 8, keys 16b + 2t (+ 1), and 8 on
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                uint32_t h[4];
                                e2m1x8_f16(vf[2 * odd + i], h);
                                const uint32_t s0 = in_low(vscale[i][0][c2], odd), s1 = in_high(vscale[i][1][c2], odd);
#pragma unroll
                                for (int j = 0; j < 2; ++j)
#pragma unroll
                                    for (int r = 0; r < 2; ++r) a[r][2 * i + j] = hfma2(both(h[j], r), s0, hmul2(both(h[2 + j], r), s1));
                            }
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int r = 0; r < 2; ++r) mma16816<true>(o[n][4 * c2 + 2 * odd + r], a[r], pb[n][b][0], pb[n][b][1]);
                        }
                    }
                }
            }
        }
        copy_wait<0>();
        __syncwarp();

        // ---- the four warps' results join
        const float vs = p.v_scale[pc.h];
        float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float sum = l[n][r];
#pragma unroll
                for (int x = 4; x < 32; x *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                const int m = 8 * n + 2 * t + r;
                if (g == 0) {
                    s_m[w][m] = mx[n][r];
                    s_l[w][m] = sum;
                }
#pragma unroll
                for (int c = 0; c < DT / 32; ++c)
                    *reinterpret_cast<float4*>(mine + m * Sh::kLd + 32 * c + 4 * g) =
                        make_float4(o[n][2 * c][r], o[n][2 * c + 1][r], o[n][2 * c][2 + r], o[n][2 * c + 1][2 + r]);
            }
        __syncthreads();
        const bool whole = pc.whole();
        if (tid < M) {
            // a row's maximum and sum, and each warp's factor in its output (the values' scale and, where
            // this is the whole, the sum with it)
            const float c = s_qs[tid];
            float big = kNone, sum = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) big = fmaxf(big, s_m[i][tid]);
            // The maximum is m c as a float32 from here on; what that leaves out goes into the sum and the output
            // (up to 2^63 either way, which scores below 2^30 stay within).
            const float top = big == kNone ? ninf : big * c;
            const float rest = top == ninf ? -kShift : fminf(fmaxf(fmaf(big, c, -top), -63.f), 63.f) - kShift;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) sum += s_l[i][tid] * fast_exp2(fmaf(s_m[i][tid] - big, c, rest));
            const float f = !whole ? vs : sum != 0.f ? vs / sum : 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) s_m[i][tid] = f * fast_exp2(fmaf(s_m[i][tid] - big, c, rest));
            if (tid < valid) {
                if (!whole) {
                    reinterpret_cast<float2*>(p.part_ml)[part_place(blockIdx.x, pc.u0 == 0) * M + tid] = make_float2(top, sum);
                } else if (p.lse != nullptr) {
                    const int qi = pc.tile * M + tid;
                    p.lse[(static_cast<int64_t>(pc.r.row0) + qi / p.G) * p.Hq + pc.h * p.G + qi % p.G] = lse_of(top, sum);
                }
            }
        }
        __syncthreads();
        constexpr int kCols = DT / 4;                        // threads of a row
        const int d = tid % kCols * 4;
        float* part = p.part_o + part_place(blockIdx.x, pc.u0 == 0) * M * p.D + d;
#pragma unroll 2
        for (int m = tid / kCols; m < (d < p.D ? valid : 0); m += kThreads / kCols) {
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
                store_four(part + m * p.D, x);
            }
        }
        if (!whole && part_done(p, pc, st, &s_flag, tid, [] { __syncthreads(); }))
            join_parts<__nv_bfloat16, M, kThreads>(p, pc, st, s_row, tid, [] { __syncthreads(); });
        __syncthreads();
    }
    if (blockIdx.x == 0) head_cleared();
}

template <int DT, int NT>
dspark_status_t launch_mma4(const Args& p, cudaStream_t s) {
    using Sh = Mma4Shape<DT, NT>;
    static OncePerDevice once;
    const int dev = current_device();
    if (once.run(dev, [] {
            return cudaFuncSetAttribute(attend_mma4<DT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
        }) != cudaSuccess)
        return DSPARK_ERR_CUDA;
    const int grid = grid_for(sm_count(dev) * Sh::kPerSm, Sh::M);
    if (grid < 1) return DSPARK_ERR_CUDA;
    return launch_cleared(p.status, kHeadBytes, attend_mma4<DT, NT>, dim3(grid), Sh::kThreads, Sh::kSmem, s, p);
}

}  // namespace attn
}  // namespace dspark
