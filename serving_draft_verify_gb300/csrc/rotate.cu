// dspark_rotate and dspark_rotate_write_kv: rotary positions, and a step's rows stored in the same pass.
//
// Pair i of a head (elements i and i + rot / 2, or 2i and 2i + 1) at position n turns by n freq[i]:
//   y1 = m (x1 cos a - x2 sin a),  y2 = m (x2 cos a + x1 sin a).
//
// The angle.  n freq in float32 is off by 2^-24 of itself, which at position 10^6 is a sixteenth of a
// radian.  Here freq / 2 pi is a 64-bit fraction of a turn, formed with integers from freq's 24 bits
// (wrong by 2^-64 at most for |freq| < 4, and by |freq| / 4 of that above), so that n times it, modulo 2^64, is the angle modulo
// a turn to 2^-33;
// the nearest quarter turn is taken off before anything is rounded to float32.
//
// Bound by memory: every element is read once and written once.  A block has a few rows: its threads
// first make the rows' cosines and sines, then each has one place of a head (`unit`: two pieces of kSub
// elements that hold whole pairs, so that a call in place needs no exchange) and goes over the heads
// with it.  In a graph, one call after the other: 16384 rows of 40 heads of 128, bf16: 54 us for 336 MB (6.2 TB/s; 52 by the
// profiler, without the gap between launches; 55 to 56 through the Python binding), float32 8192 rows of them 54; 16384 rows of
// 32 heads on 8 with keys and values stored in 4 bits: 72 us for 354 MB (4.9 TB/s), issuing in 57 % of the cycles, its warps
// waiting for memory (3.9 of the 11 cycles between two instructions of one), then for shared memory and for fixed latency
// (1.8 each); keys and values alone to 4 bits, not rotated, 24 us (86 MB, 3.6 TB/s), issuing in 62 %, waits of 2.2 cycles of 10 for
// memory, 2.1 for fixed latency, 1.4 at the barrier behind the rows' places; float32 to 4 bits (8192 rows) 59 us.
#include <cmath>

#include "launch.cuh"
#include "rotate.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxRows = 4;                     // of a block
constexpr int kItems = 2;                       // heads in flight where they stand in one line over the rows
constexpr int kSub = 8;                         // elements of a piece
constexpr int kMaxPairs = 128;                  // of a head
constexpr int64_t kAlone = 256;                 // rows up to which one launch does, as in kv_write.cu

// kNone: queries alone; kFew: the same with fewer heads than a block has groups of threads.
enum Cache { kNone, kFew, kSame, kE4m3, kE2m1 };

// freq / 2 pi as a fraction of a turn in units of 2^-64: freq = m 2^(e - 25 + 2 - 64) with the constant
// 2^66 / 2 pi.  Frequencies below 2^26; signs by the caller.
__device__ __forceinline__ uint64_t turn_of(float freq) {
    const uint32_t u = __float_as_uint(freq) & 0x7FFFFFFFu;
    const int e = static_cast<int>(u >> 23);
    const uint64_t m = e == 0 ? u : (u & 0x007FFFFFu) | 0x00800000u;
    constexpr uint64_t kTurn = 0xA2F9836E4E44152Aull;
    const uint64_t lo = m * kTurn, hi = __umul64hi(m, kTurn);
    const int down = 25 - ((e == 0 ? 1 : e) - 127);          // of the 88-bit product
    if (down <= 0) return lo;
    if (down < 64) return (lo >> down) | (hi << (64 - down));
    return down < 128 ? hi >> (down - 64) : 0;
}
// Cosine and sine of a fraction of a turn.
__device__ __forceinline__ float2 cos_sin(uint64_t a) {
    const uint32_t q = static_cast<uint32_t>((a + (1ull << 61)) >> 62);       // the nearest quarter
    const int64_t rest = static_cast<int64_t>(a - (static_cast<uint64_t>(q) << 62));
    float s, c;
    sincospif(static_cast<float>(rest) * 0x1p-63f, &s, &c);                  // half turns
    const float2 r = (q & 1) ? make_float2(-s, c) : make_float2(c, s);
    return (q & 2) ? make_float2(-r.x, -r.y) : r;
}

// Heads of queries in flight and blocks an SM asked for.  At seven blocks (72 registers) bf16 rows to 4 bits spill 28 bytes of
// stores and 80 of loads (interleaved 44 and 60), to 8 bits 8 and 36 (4 and 4); float32 ones to 4 bits at five blocks, interleaved,
// 20 and 36: 1 % of the instructions where it was counted (the first).  16384 rows of 32 heads on 8 of 128, bf16, to 4 bits, us:
// 72 with 2 heads and 7 blocks, 75 with 3 and 6, 82 with 3 and 5, 95 with 3 heads and no blocks asked for; rotation alone takes
// three heads and what registers it likes (40 heads 54, with 2 heads 57); float32 60 with 3 and 5, 70 with 2 and 7.
// Few heads, 16384 rows of 8: 14.5 with 8 blocks, 16.3 without asking for any, and 25.7 a row at a time.
template <typename T, Cache kCache>
constexpr int kHeads = kCache == kNone || sizeof(T) == 4 ? 3 : 2;
template <typename T, Cache kCache>
constexpr int kBlocks = kCache == kNone ? 1 : sizeof(T) == 4 ? 5 : kCache == kFew ? 8 : 7;

// kN adjacent elements, as they lie in memory.
template <typename T, int kN>
struct Piece {
    uint4 w[kN * sizeof(T) / 16];
    __device__ __forceinline__ void load(const void* p) {
#pragma unroll
        for (int i = 0; i < kN * static_cast<int>(sizeof(T)) / 16; ++i) w[i] = *(static_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void store(void* p) const {
#pragma unroll
        for (int i = 0; i < kN * static_cast<int>(sizeof(T)) / 16; ++i) *(static_cast<uint4*>(p) + i) = w[i];
    }
    __device__ __forceinline__ void floats(float* f) const {
#pragma unroll
        for (int i = 0; i < kN * static_cast<int>(sizeof(T)) / 16; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 2) {
                    f[8 * i + 2 * j] = bf16lo(u[j]);
                    f[8 * i + 2 * j + 1] = bf16hi(u[j]);
                } else {
                    f[4 * i + j] = __uint_as_float(u[j]);
                }
            }
        }
    }
    __device__ __forceinline__ void set(const float* f) {
#pragma unroll
        for (int i = 0; i < kN * static_cast<int>(sizeof(T)) / 16; ++i) {
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 2) {
                    const __nv_bfloat162 two = __floats2bfloat162_rn(f[8 * i + 2 * j], f[8 * i + 2 * j + 1]);
                    u[j] = *reinterpret_cast<const uint32_t*>(&two);
                } else {
                    u[j] = __float_as_uint(f[4 * i + j]);
                }
            }
            w[i] = make_uint4(u[0], u[1], u[2], u[3]);
        }
    }
};

// Two pieces turned: pairs (j, kSub + j) of them, or adjacent elements.
template <bool kInter>
__device__ __forceinline__ void turn_floats(float* f, const float2* turn) {
#pragma unroll
    for (int j = 0; j < kSub; ++j) {
        const int j1 = kInter ? 2 * j : j, j2 = kInter ? 2 * j + 1 : kSub + j;
        const float x1 = f[j1], x2 = f[j2];
        f[j1] = fmaf(x1, turn[j].x, -x2 * turn[j].y);
        f[j2] = fmaf(x2, turn[j].x, x1 * turn[j].y);
    }
}
template <typename T, bool kInter>
__device__ __forceinline__ void turn_pieces(Piece<T, kSub>* x, const float2* turn) {
    float f[2 * kSub];
    x[0].floats(f);
    x[1].floats(f + kSub);
    turn_floats<kInter>(f, turn);
    x[0].set(f);
    x[1].set(f + kSub);
}

template <typename T, Cache kCache, bool kInter>
__global__ void __launch_bounds__(kThreads, (kBlocks<T, kCache>)) rotate_rows(const __grid_constant__ RotateArgs p) {
    __shared__ __align__(16) float2 s_turn[kMaxRows][kMaxPairs];
    __shared__ int64_t s_to[kMaxRows];                       // a row's place in its page, -1: none
    __shared__ int s_block[kMaxRows];
    __shared__ bool s_live[kMaxRows];
    constexpr int kHeads = dspark::kHeads<T, kCache>;
    const int tid = threadIdx.x, half = p.rot / 2;
    // Where there are both, every second block has queries, the others keys and values: the former's
    // bytes move while the latter's arithmetic runs (16384 rows to 4 bits: 79 us where a block did both).
    const bool mixed = kCache > kFew && p.Hq > 0, stores = kCache > kFew && (!mixed || (blockIdx.x & 1) != 0);
    const int64_t row0 = static_cast<int64_t>(mixed ? blockIdx.x >> 1 : blockIdx.x) * p.rows_per_block;
    const int64_t left = p.rows - row0;
    const int n = left < p.rows_per_block ? static_cast<int>(left) : p.rows_per_block;
    // Alone, the first block clears the status and looks at the slots of all rows.
    const bool all = p.alone && blockIdx.x == 0;
    if (all && tid < 4) reinterpret_cast<uint32_t*>(p.status)[tid] = 0;
    const int u = tid % p.units, first = tid / p.units, groups = kThreads / p.units;
    const bool turned = u < p.turned;
    // the places of the unit's two pieces in a head
    const int a = turned ? (kInter ? 2 * kSub * u : kSub * u) : p.rot + 2 * kSub * (u - p.turned);
    const int b = turned && !kInter ? a + half : a + kSub;
    const int heads = stores ? 2 * p.Hkv : p.Hq;             // keys', then values'; or queries'
    // Heads of all the block's rows in one line, kItems at a time, the first loaded while the angles are made:
    // keys and values, and queries with fewer heads than there are groups of threads, which would have
    // one at a time (16384 rows of 12 heads on 1: 38 us, a row at a time 43; 32 heads on 8: 82 and 72).
    struct Batch {
        Piece<T, kSub> x[kItems][2];
        int r[kItems], h[kItems];
    };
    int r_next = first < groups ? 0 : n, h_next = first;
    auto load = [&](Batch& t) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            while (h_next >= heads) {
                h_next -= heads;
                ++r_next;
            }
            const int r = r_next, h = h_next;
            t.r[i] = r;
            t.h[i] = h;
            h_next += groups;
            if (r >= n) continue;
            const bool is_v = h >= p.Hkv;
            const T* from = static_cast<const T*>(!stores ? p.q : is_v ? p.v : p.k) +
                            (row0 + r) * (!stores ? p.q_stride : is_v ? p.v_stride : p.k_stride) + (stores && is_v ? h - p.Hkv : h) * p.D;
            t.x[i][0].load(from + a);
            t.x[i][1].load(from + b);
        }
    };
    Batch now;
    const bool rowwise = kCache == kNone || (kCache != kFew && !stores && heads > groups);
    if (!rowwise) load(now);
    bool past = false;
    for (int r = tid; r < (all && p.slot != nullptr ? static_cast<int>(p.rows) : n); r += kThreads) {
        const bool live = p.position == nullptr || p.position[row0 + r] >= 0;
        int64_t slot = p.slot != nullptr ? p.slot[row0 + r] : -1;
        int block = 0;
        if (slot >= p.slots && live) past = true;
        if (!live || slot >= p.slots) slot = -1;
        if (slot >= 0) {
            block = static_cast<int>((slot >> 32) == 0 ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.page) : slot / p.page);
            slot -= static_cast<int64_t>(block) * p.page;
        }
        if (r < n) {
            s_live[r] = live;
            s_to[r] = slot;
            s_block[r] = block;
        }
    }
    for (int e = tid; e < n * half; e += kThreads) {
        const int r = e / half, i = e - r * half;
        const float f = __ldg(p.freq + i);
        const int32_t at = p.position[row0 + r];
        const float2 cs = cos_sin(turn_of(f) * static_cast<uint64_t>(static_cast<uint32_t>(at < 0 ? 0 : at)));
        const bool odd = !(fabsf(f) < 0x1p26f);               // no angle: not a number
        s_turn[r][i] = odd ? make_float2(__uint_as_float(0x7fffffffu), __uint_as_float(0x7fffffffu))
                           : make_float2(cs.x * p.magnitude, ((f < 0.f) != p.transposed ? -cs.y : cs.y) * p.magnitude);
    }
    __syncthreads();
    if (past && (all || !p.alone)) tell(p.status, DSPARK_ERR_DEVICE_CHECK, 1);

    if (rowwise) {
        // ---- queries: a row at a time, so that its angles stay in registers
        for (int r = 0; r < n; ++r) {
            if (!s_live[r] || first >= groups) continue;
            float2 turn[kSub];
            if (turned) {
#pragma unroll
                for (int j = 0; j < kSub; j += 2)
                    *reinterpret_cast<float4*>(turn + j) = *reinterpret_cast<const float4*>(&s_turn[r][kSub * u + j]);
            }
            const T* from = static_cast<const T*>(p.q) + (row0 + r) * p.q_stride;
            T* out = static_cast<T*>(p.out) + (row0 + r) * p.out_stride;
            for (int h0 = first; h0 < heads; h0 += kHeads * groups) {
                Piece<T, kSub> x[kHeads][2];
#pragma unroll
                for (int i = 0; i < kHeads; ++i) {
                    const int h = h0 + i * groups;
                    if (h >= heads) continue;
                    x[i][0].load(from + h * p.D + a);
                    x[i][1].load(from + h * p.D + b);
                }
#pragma unroll
                for (int i = 0; i < kHeads; ++i) {
                    const int h = h0 + i * groups;
                    if (h >= heads) continue;
                    if (turned) turn_pieces<T, kInter>(x[i], turn);
                    x[i][0].store(out + h * p.D + a);
                    x[i][1].store(out + h * p.D + b);
                }
            }
        }
    } else if constexpr (kCache != kNone) {
        int of = -1;                                         // the head whose scale these are
        float scale = 0.f, sixth = 0.f;
        while (now.r[0] < n) {
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const int r = now.r[i], h = now.h[i];
                if (r >= n || !(stores ? s_to[r] >= 0 : s_live[r])) continue;
                const int64_t to = s_to[r];
                const bool is_v = h >= p.Hkv, as_is = (stores && is_v) || !turned;
                Piece<T, kSub>* x = now.x[i];
                float2 turn[kSub];
                if (!as_is) {
#pragma unroll
                    for (int j = 0; j < kSub; j += 2)
                        *reinterpret_cast<float4*>(turn + j) = *reinterpret_cast<const float4*>(&s_turn[r][kSub * u + j]);
                }
                if (!stores) {
                    T* out = static_cast<T*>(p.out) + (row0 + r) * p.out_stride + h * p.D;
                    if (!as_is) turn_pieces<T, kInter>(x, turn);
                    x[0].store(out + a);
                    x[1].store(out + b);
                    continue;
                }
                const int head = is_v ? h - p.Hkv : h;
                const int64_t page = static_cast<int64_t>(s_block[r]) * p.Hkv + head;
                if constexpr (kCache == kSame) {
                    T* cache = static_cast<T*>(is_v ? p.vc : p.kc) + (page * p.page + to) * p.D;
                    if (!as_is) turn_pieces<T, kInter>(x, turn);
                    x[0].store(cache + a);
                    x[1].store(cache + b);
                    continue;
                }
                float f[2 * kSub];
                x[0].floats(f);
                x[1].floats(f + kSub);
                if (!as_is) turn_floats<kInter>(f, turn);
                if constexpr (kCache == kE4m3) {
                    uint8_t* cache = static_cast<uint8_t*>(is_v ? p.vc : p.kc) + (page * p.page + to) * p.D;
                    const float scale = __ldg((is_v ? p.v_scale : p.k_scale) + head), inv = __fdiv_rn(1.f, scale), margin = margin_of(scale);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t w[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float* y = f + 8 * j + 4 * k;
                            w[k] = stored(y[0], y[1], scale, inv, margin) | (stored(y[2], y[3], scale, inv, margin) << 16);
                        }
                        *reinterpret_cast<uint2*>(cache + (j == 0 ? a : b)) = make_uint2(w[0], w[1]);
                    }
                } else if constexpr (kCache == kE2m1) {
                    uint8_t* cache = static_cast<uint8_t*>(is_v ? p.vc : p.kc) + page * p.g.whole;
                    if (h != of) of = h, scale = __ldg((is_v ? p.v_scale : p.k_scale) + head), sixth = __frcp_rn(6.f * scale);
                    uint8_t *codes = cache + to * p.g.code, *scales = cache + p.g.codes + to * p.g.scale;
                    // Two pieces side by side are a block of 16; two that lie apart are halves of two, whose other
                    // halves the neighbouring thread has (heads have an even number of units): the first thread
                    // makes the scale of the first block, the second that of the other.
                    float big = magnitude8(f), inv[2];
                    const float big2 = magnitude8(f + 8);
                    if (kInter || !turned) {
                        const Scale4 s = scale4(magnitude3(big, big2, 0.f), scale, sixth);
                        inv[0] = inv[1] = s.inv;
                        scales[a / 16] = static_cast<uint8_t>(s.byte);
                    } else {
                        const uint32_t pair = 3u << (tid & 30);
                        const bool second = (tid & 1) != 0;
                        const float theirs = __shfl_xor_sync(pair, second ? big : big2, 1);
                        const Scale4 s = scale4(magnitude3(second ? big2 : big, theirs, 0.f), scale, sixth);
                        const float other = __shfl_xor_sync(pair, s.inv, 1);
                        inv[0] = second ? other : s.inv;
                        inv[1] = second ? s.inv : other;
                        scales[(second ? b : a) / 16] = static_cast<uint8_t>(s.byte);
                    }
                    *reinterpret_cast<uint32_t*>(codes + a / 2) = codes8(f, inv[0]);
                    *reinterpret_cast<uint32_t*>(codes + b / 2) = codes8(f + 8, inv[1]);
                }
            }
            load(now);
        }
    }
    if (blockIdx.x == 0) head_cleared();
}

template <typename T, bool kInter>
void (*kernel_of(Cache c))(RotateArgs) {
    switch (c) {
        case kNone: return rotate_rows<T, kNone, kInter>;
        case kFew: return rotate_rows<T, kFew, kInter>;
        case kSame: return rotate_rows<T, kSame, kInter>;
        case kE4m3: return rotate_rows<T, kE4m3, kInter>;
        default: return rotate_rows<T, kE2m1, kInter>;
    }
}

// Whether rows of `width` elements at `stride` from x and rows of `width2` at `stride2` from y share memory.
bool rows_meet(const void* x, int64_t stride, int64_t width, const void* y, int64_t stride2, int64_t width2, int64_t rows,
               int64_t size) {
    if (rows == 0 || width == 0 || width2 == 0) return false;
    const int64_t a = static_cast<int64_t>(reinterpret_cast<uintptr_t>(x)), b = static_cast<int64_t>(reinterpret_cast<uintptr_t>(y));
    if (a + ((rows - 1) * stride + width) * size <= b || b + ((rows - 1) * stride2 + width2) * size <= a) return false;
    if (stride != stride2) return true;
    int64_t d = (b - a) % (stride * size);                   // slices of one buffer
    if (d < 0) d += stride * size;
    return d < width * size || d + width2 * size > stride * size;
}

// What every call checks of the rotation; `unit`: elements that a thread's pieces come to.
bool rotation_ok(int64_t rows, int D, int rot, int interleaved, int unit, const void* position, const void* freq,
                 float magnitude) {
    return D >= unit && D <= 256 && D % unit == 0 && rot >= unit && rot <= D && rot % unit == 0 &&
           (interleaved == 0 || interleaved == 1) && (rows == 0 || position != nullptr) && freq != nullptr && magnitude - magnitude == 0.f;
}
bool rows_ok(int64_t rows, int64_t width, dspark_dtype_t dt, const void* x, int64_t stride) {
    return stride >= width && stride % (dt == DSPARK_BF16 ? 8 : 4) == 0 && aligned16(x) && (rows == 0 || x != nullptr);
}

}  // namespace

dspark_status_t launch_rotate(RotateArgs p, dspark_dtype_t dt, dspark_dtype_t cache_dt, cudaStream_t s) {
    const Cache c = p.Hkv == 0 ? (p.Hq <= kThreads / (p.D / 16) ? kFew : kNone) : cache_dt == DSPARK_E2M1 ? kE2m1 : cache_dt == DSPARK_E4M3 ? kE4m3 : kSame;
    p.units = p.D / 16;
    p.turned = p.rot / 16;
    p.g = page4_of(p.page, p.D);
    p.rows_per_block = kMaxRows;
    while (p.rows_per_block > 1 && (p.rows + p.rows_per_block - 1) / p.rows_per_block < 2 * sm_count(current_device()))
        p.rows_per_block /= 2;
    p.alone = p.slot == nullptr || p.rows <= kAlone;
    const unsigned grid = static_cast<unsigned>((p.rows + p.rows_per_block - 1) / p.rows_per_block) * (p.Hq > 0 && p.Hkv > 0 ? 2 : 1);
    void (*kernel)(RotateArgs) = dt == DSPARK_BF16
                                     ? (p.interleaved ? kernel_of<__nv_bfloat16, true>(c) : kernel_of<__nv_bfloat16, false>(c))
                                     : (p.interleaved ? kernel_of<float, true>(c) : kernel_of<float, false>(c));
    if (p.alone) {
        kernel<<<grid, kThreads, 0, s>>>(p);
        return launch_status();
    }
    return launch_cleared(p.status, kStatusBytes, kernel, dim3(grid), kThreads, 0, s, p);
}

}  // namespace dspark

extern "C" dspark_status_t dspark_rotary_frequencies(int rot, double base, dspark_rotary_scaling_t scaling, double factor,
                                                     double original, double low, double high, float* freq,
                                                     float* magnitude) {
    using std::exp;
    using std::log;
    if (rot < 2 || rot > 256 || rot % 2 != 0 || freq == nullptr || !(base > 1.0) || !std::isfinite(base) ||
        scaling < DSPARK_ROTARY_PLAIN || scaling > DSPARK_ROTARY_BANDS)
        return DSPARK_ERR_INVALID_ARGUMENT;
    const bool ranged = scaling == DSPARK_ROTARY_RAMP || scaling == DSPARK_ROTARY_BANDS;
    if (scaling != DSPARK_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return DSPARK_ERR_INVALID_ARGUMENT;
    if (ranged && (!(original > 0.0) || !std::isfinite(original) || !(low > 0.0) || !(high > low) || !std::isfinite(high)))
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (scaling == DSPARK_ROTARY_BASE && rot == 2) return DSPARK_ERR_INVALID_ARGUMENT;
    const double turn = 6.283185307179586476925;
    // of the base in use, which itself may leave the doubles
    const double log_base = log(base) + (scaling == DSPARK_ROTARY_BASE ? rot / (rot - 2.0) * log(factor) : 0.0);
    auto pair_with = [&](double turns) { return rot * log(original / (turns * turn)) / (2.0 * log(base)); };
    double first = 0.0, last = 0.0;
    if (scaling == DSPARK_ROTARY_RAMP) {
        first = std::floor(pair_with(high)), last = std::ceil(pair_with(low));
        first = first < 0.0 ? 0.0 : first, last = last > rot - 1.0 ? rot - 1.0 : last;
        if (last <= first) last = first + 0.001;
    }
    for (int i = 0; i < rot / 2; ++i) {
        const double f = exp(-2.0 * i / rot * log_base);
        double keep = 1.0;                                   // of f; the rest is f / factor
        if (scaling == DSPARK_ROTARY_LINEAR) keep = 0.0;
        if (scaling == DSPARK_ROTARY_RAMP) keep = 1.0 - (i - first) / (last - first);
        if (scaling == DSPARK_ROTARY_BANDS) keep = (original * f / turn - low) / (high - low);
        keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
        freq[i] = static_cast<float>(keep == 1.0 ? f : f * keep + f / factor * (1.0 - keep));
    }
    if (magnitude != nullptr) *magnitude = scaling == DSPARK_ROTARY_RAMP ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.f;
    return DSPARK_OK;
}

extern "C" size_t dspark_rotate_workspace_size(void) { return dspark::kStatusBytes; }

extern "C" dspark_status_t dspark_rotate(int64_t rows, int heads, int D, int rot, int interleaved, int transposed,
                                         dspark_dtype_t dt, const void* x, int64_t x_stride, const int32_t* position,
                                         const float* freq, float magnitude, void* out, int64_t out_stride,
                                         void* workspace, size_t workspace_bytes, dspark_stream_t stream) {
    using namespace dspark;
    if (rows < 0 || rows > 0x7fffffffll || heads < 1 || heads > 4096 || (dt != DSPARK_BF16 && dt != DSPARK_F32) ||
        (transposed != 0 && transposed != 1) || !rotation_ok(rows, D, rot, interleaved, 16, position, freq, magnitude))
        return DSPARK_ERR_INVALID_ARGUMENT;
    const int64_t width = static_cast<int64_t>(heads) * D, size = dt == DSPARK_BF16 ? 2 : 4;
    if (!rows_ok(rows, width, dt, x, x_stride) || !rows_ok(rows, width, dt, out, out_stride)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (!(x == out && x_stride == out_stride) && rows_meet(x, x_stride, width, out, out_stride, width, rows, size))
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (workspace == nullptr || !aligned256(workspace)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < dspark_rotate_workspace_size()) return DSPARK_ERR_WORKSPACE_TOO_SMALL;
    clear_stale_error();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) return clear_status(workspace, s);
    RotateArgs p{};
    p.rows = rows, p.q_stride = x_stride, p.out_stride = out_stride, p.Hq = heads, p.D = D, p.rot = rot, p.page = 1;
    p.interleaved = interleaved != 0, p.transposed = transposed != 0, p.q = x, p.position = position, p.freq = freq;
    p.magnitude = magnitude, p.out = out, p.status = static_cast<StatusBlock*>(workspace);
    return launch_rotate(p, dt, dt, s);
}

extern "C" size_t dspark_rotate_write_kv_workspace_size(void) { return dspark::kStatusBytes; }

extern "C" dspark_status_t dspark_rotate_write_kv(
    int64_t rows, int Hq, int Hkv, int D, int rot, int interleaved, int page, int num_blocks, dspark_dtype_t dt,
    dspark_dtype_t cache_dt, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
    int64_t v_stride, const int32_t* position, const float* freq, float magnitude, const int64_t* slot,
    const float* k_scale, const float* v_scale, void* q_out, int64_t q_out_stride, void* k_cache, void* v_cache,
    void* workspace, size_t workspace_bytes, dspark_stream_t stream) {
    using namespace dspark;
    const bool scaled = cache_dt == DSPARK_E4M3 || cache_dt == DSPARK_E2M1;
    if (rows < 0 || rows > 0x7fffffffll || Hq < 0 || Hq > 4096 || Hkv < 1 || Hkv > 1024 || page < 1 || num_blocks < 1 ||
        (dt != DSPARK_BF16 && dt != DSPARK_F32) || (cache_dt != dt && !scaled) ||
        !rotation_ok(rows, D, rot, interleaved, cache_dt == DSPARK_E2M1 ? 32 : 16, position, freq, magnitude))
        return DSPARK_ERR_INVALID_ARGUMENT;
    const int64_t width = static_cast<int64_t>(Hkv) * D, qw = static_cast<int64_t>(Hq) * D, size = dt == DSPARK_BF16 ? 2 : 4;
    if (!rows_ok(rows, width, dt, k, k_stride) || !rows_ok(rows, width, dt, v, v_stride) || (rows > 0 && slot == nullptr) ||
        k_cache == nullptr || v_cache == nullptr || !aligned16(k_cache) || !aligned16(v_cache) ||
        (scaled && (k_scale == nullptr || v_scale == nullptr)))
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (Hq > 0 && (!rows_ok(rows, qw, dt, q, q_stride) || !rows_ok(rows, qw, dt, q_out, q_out_stride) ||
                   (!(q == q_out && q_stride == q_out_stride) && rows_meet(q, q_stride, qw, q_out, q_out_stride, qw, rows, size)) ||
                   rows_meet(k, k_stride, width, q_out, q_out_stride, qw, rows, size) ||
                   rows_meet(v, v_stride, width, q_out, q_out_stride, qw, rows, size)))
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (cache_dt == DSPARK_E2M1 && static_cast<int64_t>(page) * D > 0x7fffffffll - 1024) return DSPARK_ERR_UNSUPPORTED;
    if (workspace == nullptr || !aligned256(workspace)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < dspark_rotate_write_kv_workspace_size()) return DSPARK_ERR_WORKSPACE_TOO_SMALL;
    clear_stale_error();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) return clear_status(workspace, s);
    RotateArgs p{};
    p.rows = rows, p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride, p.out_stride = q_out_stride;
    p.slots = static_cast<int64_t>(num_blocks) * page, p.Hq = Hq, p.Hkv = Hkv, p.D = D, p.rot = rot, p.page = page;
    p.interleaved = interleaved != 0, p.q = q, p.k = k, p.v = v, p.position = position, p.freq = freq;
    p.magnitude = magnitude, p.slot = slot, p.k_scale = k_scale, p.v_scale = v_scale, p.out = q_out, p.kc = k_cache;
    p.vc = v_cache, p.status = static_cast<StatusBlock*>(workspace);
    return launch_rotate(p, dt, cache_dt, s);
}
