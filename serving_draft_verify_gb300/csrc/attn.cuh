// Shared parts of dspark_paged_attention's kernels: the work list and how it is
// divided over the GPU, and the joining of parts.
//
// Mathematics.  For query row i (0-based) of request b, at position len_b + i, and
// query head hq of key head h, with scores s_j = scale q . k_j over the visible keys
// j <= len_b + i (j > len_b + i - window with a window):
//   lse = ln sum_j exp(s_j),  out = sum_j exp(s_j - lse) v_j.
// A part of the keys gives m = max s_j, l = sum exp(s_j - m), o = sum exp(s_j - m)
// v_j; two parts join as m = max(m1, m2), l = sum_i l_i exp(m_i - m), likewise o.
// Scores are kept in units of log 2, so that exp is ex2.
//
// Work list.  The query rows of one key head (row i, head g of its group; index
// i G + g) are cut into tiles of M, and the keys a tile can see into units of KT.
// All units of all (request, key head, tile) segments stand in one line, and block c
// of n (n no more than W) takes units [c W / n, (c + 1) W / n): an even division whatever the lengths
// are, found by every block from the lengths on the device.  A segment that no
// block holds whole is joined by the last of its blocks to finish (a counter, nobody
// waits), its parts always in the order of the keys, so results do not depend on
// who came last.
#pragma once

#include "launch.cuh"

namespace dspark {
namespace attn {

struct Args {
    int B, Hq, Hkv, G, D, page, max_blocks, num_blocks, max_rows, window;
    int64_t rows, ld_table, q_stride;
    const void* q;
    const int32_t *row_offset, *length, *table;
    const void *kc, *vc;
    const float *k_scale, *v_scale;
    float scale_log2;                 // scale * log2(e)
    void* out;
    float* lse;
    StatusBlock* status;
    uint32_t* counters;               // [grid] parts that are done of the segment that starts in a block's range
    float* part_ml;                   // [2 grid][M][2]
    float* part_o;                    // [2 grid][M][D]
};

constexpr int kMaxGrid = 1024;
constexpr size_t kCounterBytes = kMaxGrid * 4;
constexpr int kMaxPartRows = 40960;         // query rows of all places: 2 grid M of any launch

constexpr size_t kHeadBytes = kStatusBytes + kCounterBytes;      // what starts at zero

// Blocks of a launch: as many as can be resident, so that the even division is one wave.
inline int grid_for(int resident, int M) {
    int n = resident < kMaxGrid ? resident : kMaxGrid;
    return n < kMaxPartRows / (2 * M) ? n : kMaxPartRows / (2 * M);
}

struct Request {
    int row0, n, len;                 // first row, rows, keys before the step
};
// What the lengths say about request b; an inconsistent one has no rows.
__device__ __forceinline__ Request request_of(const Args& p, int b, bool report) {
    Request r;
    r.row0 = p.row_offset[b];
    const int64_t n = static_cast<int64_t>(p.row_offset[b + 1]) - r.row0;
    r.len = p.length[b];
    const int64_t cap = static_cast<int64_t>(p.max_blocks) * p.page;
    const bool ok = n >= 0 && n <= p.max_rows && r.row0 >= 0 && r.row0 + n <= p.rows && r.len >= 0 && r.len + n <= cap;
    if (!ok && report) tell(p.status, DSPARK_ERR_DEVICE_CHECK, 1);
    r.n = ok ? static_cast<int>(n) : 0;
    return r;
}
// The keys [seen, hi) that tile t of a request's query rows can see, and its units.  Nothing is read
// for the keys from lo to seen: pages that a window has left behind may be gone.
struct Span {
    int lo, hi, seen;                 // lo: the unit's border at or before seen
    __device__ __forceinline__ int units(int KT) const { return hi > lo ? (hi - lo + KT - 1) / KT : 1; }
};
template <int M, int KT>
__device__ __forceinline__ Span span_of(const Args& p, const Request& r, int t) {
    const int first = t * M / p.G;
    const int last = (min(static_cast<int64_t>(t + 1) * M, static_cast<int64_t>(r.n) * p.G) - 1) / p.G;
    Span s;
    s.hi = r.len + last + 1;
    s.seen = p.window > 0 ? max(0, r.len + first - p.window + 1) : 0;
    s.lo = s.seen / KT * KT;
    return s;
}
template <int M>
__device__ __forceinline__ int tiles_of(const Args& p, const Request& r) {
    return static_cast<int>((static_cast<int64_t>(r.n) * p.G + M - 1) / M);
}
// A request with the units of one of its key heads.  One copy of the code for all that ask: a
// block of a short call runs most of its instructions once, and fetching them is what it
// waits for.
struct Asked {
    Request r;
    int64_t units;
};
template <int M, int KT>
__device__ __noinline__ Asked ask(const Args& p, int b, bool report) {
    Asked a;
    a.r = request_of(p, b, report);
    a.units = 0;
    const int nt = tiles_of<M>(p, a.r);
#pragma unroll 1
    for (int t = 0; t < nt; ++t) a.units += span_of<M, KT>(p, a.r, t).units(KT);
    return a;
}

// a / b for a >= 0, b > 0; the 64-bit division only where a needs it.
__device__ __forceinline__ int64_t div_pos(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// The block's first unit: request, and units into it; found by all threads together.
// scratch: 38 words of 8 bytes.
struct Start {
    int64_t total, first, last;       // units in all, and this block's [first, last)
    int grid;                         // blocks that have units
    int b;
    int64_t into;                     // units before `first` in request b
    Asked a;                          // request b
};
template <int M, int KT, int kThreads>
__device__ __forceinline__ Start find_start(const Args& p, long long* scratch) {
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    long long mine = 0;
    Asked a{};
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        a = ask<M, KT>(p, b, blockIdx.x == 0);
        mine += p.Hkv * a.units;
    }
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) scratch[w] = inc;
    __syncthreads();
    long long before = 0, total = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
        if (i < w) before += scratch[i];
        total += scratch[i];
    }
    const long long at = before + inc - mine;
    Start s;
    s.total = total;
    // two units a block at least where units are short: a part costs its joining more than a unit does
    const long long most = M >= 128 ? total : (total + 1) / 2;
    s.grid = most < gridDim.x ? static_cast<int>(most) : static_cast<int>(gridDim.x);
    const int64_t c = blockIdx.x, n = s.grid;
    s.first = c < n ? div_pos(total * c, n) : total;
    s.last = c < n ? div_pos(total * (c + 1), n) : total;
    if (at <= s.first && s.first < at + mine) {
        long long u = at;
        int b = b0;
#pragma unroll 1
        for (; b < b1; ++b) {
            if (b1 - b0 > 1) a = ask<M, KT>(p, b, false);
            if (s.first < u + p.Hkv * a.units) break;
            u += p.Hkv * a.units;
        }
        scratch[32] = b;
        scratch[33] = s.first - u;
        scratch[34] = a.r.row0;
        scratch[35] = a.r.n;
        scratch[36] = a.r.len;
        scratch[37] = a.units;
    }
    __syncthreads();
    s.b = static_cast<int>(scratch[32]);
    s.into = scratch[33];
    s.a.r = Request{static_cast<int>(scratch[34]), static_cast<int>(scratch[35]), static_cast<int>(scratch[36])};
    s.a.units = scratch[37];
    return s;
}

// The block that holds unit u of `total` over `grid` blocks.
__device__ __forceinline__ int block_of(int64_t u, int64_t total, int grid) {
    return static_cast<int>(div_pos((u + 1) * grid - 1, total));
}

// A piece of a segment: units [u0, u1) of the segment's `units`.
struct Piece {
    Request r;
    int b, h, tile;
    Span span;
    int u0, u1, units;
    int64_t seg_first;                // the segment's first unit in the line
    __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == units; }
};

// Walks the block's units piece by piece (every thread the same way).  The first piece is looked for
// tile by tile; a further one starts the segment after the last (a prompt of 8192 rows has thousands).
template <int M, int KT>
struct Walk {
    const Args& p;
    int64_t at, last;
    int b, h, tile, u0;               // u0: units of the segment before the piece, -1 behind a segment
    Request r;
    __device__ __forceinline__ Walk(const Args& args, const Start& s)
        : p(args), at(s.first), last(s.last), b(s.b), h(0), tile(0), u0(0), r(s.a.r) {
        if (at >= last) return;
        h = static_cast<int>(div_pos(s.into, s.a.units));
        int64_t into = s.into - h * s.a.units;
        const int nt = tiles_of<M>(p, r);
#pragma unroll 1
        for (; tile + 1 < nt; ++tile) {
            const int n = span_of<M, KT>(p, r, tile).units(KT);
            if (into < n) break;
            into -= n;
        }
        u0 = static_cast<int>(into);
    }
    __device__ __forceinline__ bool next(Piece& out) {
        if (at >= last) return false;
        if (u0 < 0) {
            u0 = 0;
            if (++tile >= tiles_of<M>(p, r)) {
                tile = 0;
                if (++h >= p.Hkv) {
                    h = 0;
                    do {
                        if (++b >= p.B) return false;      // only where the lengths change under the call
                        r = request_of(p, b, false);
                    } while (r.n == 0);
                }
            }
        }
        out.r = r;
        out.b = b;
        out.h = h;
        out.tile = tile;
        out.span = span_of<M, KT>(p, r, tile);
        out.units = out.span.units(KT);
        out.u0 = u0;
        out.seg_first = at - u0;
        const int64_t left = last - at, rest = out.units - u0;
        const int n = static_cast<int>(left < rest ? left : rest);
        out.u1 = u0 + n;
        at += n;
        u0 = -1;
        return true;
    }
};

// Where a part of a segment goes: two places a block, one for the part that starts its
// segment (it is the block's last piece) and one for a part that does not.
__device__ __forceinline__ int64_t part_place(int block, bool starts) { return 2ll * block + (starts ? 1 : 0); }

// The page id at entry j of request b's table, checked.
__device__ __forceinline__ int page_id(const Args& p, int b, int j) {
    int id = __ldg(p.table + static_cast<int64_t>(b) * p.ld_table + j);
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_blocks)) {
        tell(p.status, DSPARK_ERR_DEVICE_CHECK, 2);
        id = 0;
    }
    return id;
}

// Four adjacent output elements, rounded once.
__device__ __forceinline__ void store_four(float* to, float4 x) { *reinterpret_cast<float4*>(to) = x; }
__device__ __forceinline__ void store_four(__nv_bfloat16* to, float4 x) {
    __nv_bfloat162 two[2] = {__floats2bfloat162_rn(x.x, x.y), __floats2bfloat162_rn(x.z, x.w)};
    *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(two);
}

// ln of the sum from a maximum in units of log 2 and the sum at it.
__device__ __forceinline__ float lse_of(float m, float l) { return l > 0.f || l != l ? (m + log2f(l)) * kLn2 : m; }

// Announces a stored part; true in the block that has to join the segment.  Called by the
// `tid` 0 .. n - 1 that stored it, which sync() brings together.
template <class Sync>
__device__ __forceinline__ bool part_done(const Args& p, const Piece& pc, const Start& st, int* s_flag, int tid,
                                          Sync sync) {
    const int c0 = block_of(pc.seg_first, st.total, st.grid);
    const int c1 = block_of(pc.seg_first + pc.units - 1, st.total, st.grid);
    __threadfence();
    sync();
    if (tid == 0) {
        head_cleared();
        *s_flag = atomicAdd(&p.counters[c0], 1u) == static_cast<unsigned>(c1 - c0);
    }
    sync();
    const bool join = *s_flag != 0;
    if (join) __threadfence();
    return join;
}

// Joins the parts of a segment and writes its rows: first every row's maximum and sum over the
// parts (s_row, M entries), with as many lanes a row as there are to spare, then the elements,
// four a thread from sixteen parts at a time.  The loops stay short: this code runs once a block at most, and with four pieces a thread unrolled as well it
// took longer to fetch than to run (30 parts of 4 rows: 15,000 cycles, now 8,000).
template <typename T, int M, int kThreads, class Sync>
__device__ __noinline__ void join_parts(const Args& p, Piece pc, Start st, float2* s_row, int tid, Sync sync) {
    const int c0 = block_of(pc.seg_first, st.total, st.grid);
    const int parts = block_of(pc.seg_first + pc.units - 1, st.total, st.grid) - c0 + 1;
    const int left = pc.r.n * p.G - pc.tile * M, valid = left < M ? left : M;
    const float ninf = -__uint_as_float(0x7f800000u);
    // part i of row m: place 2 (c0 + i), the first one's 2 c0 + 1
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + part_place(c0, false) * M;
    const float* po = p.part_o + part_place(c0, false) * M * p.D;
    int lanes = 1;                                           // of a row: a power of two within a warp
    while (lanes < 32 && 2 * lanes * valid <= kThreads) lanes *= 2;
#pragma unroll 1
    for (int m0 = 0; m0 < valid; m0 += kThreads / lanes) {
        const int m = m0 + tid / lanes, own = m < valid ? parts : 0;
        float mx = ninf, l = 0.f;
        auto add = [&](float m2, float l2) {
            const float big = fmaxf(mx, m2), use = big == ninf ? 0.f : big;
            l = l * fast_exp2(mx - use) + l2 * fast_exp2(m2 - use);
            mx = big;
        };
#pragma unroll 2
        for (int i = tid % lanes; i < own; i += lanes) {
            const float2 x = __ldcg(ml + (i > 0 ? 2 * i : 1) * M + m);
            add(x.x, x.y);
        }
#pragma unroll 1
        for (int o = lanes / 2; o > 0; o /= 2) add(__shfl_xor_sync(0xffffffffu, mx, o), __shfl_xor_sync(0xffffffffu, l, o));
        const float use = mx == ninf ? 0.f : mx;
        if (m < valid && tid % lanes == 0) {
            s_row[m] = make_float2(use, l);
            if (p.lse != nullptr) {
                const int qi = pc.tile * M + m;
                p.lse[(static_cast<int64_t>(pc.r.row0) + qi / p.G) * p.Hq + pc.h * p.G + qi % p.G] = lse_of(mx, l);
            }
        }
    }
    sync();
    constexpr int kC = 16;
    const int four = p.D / 4, total = valid * four;
#pragma unroll 1
    for (int e = tid; e < total; e += kThreads) {
        const int m = e / four, d = (e - m * four) * 4;
        const float use = s_row[m].x, l = s_row[m].y, inv = l != 0.f ? 1.f / l : 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int i0 = 0; i0 < parts; i0 += kC) {
            float4 x[kC];
            float f[kC];
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                const int at = (i0 + i > 0 ? 2 * (i0 + i) : 1) * M + m;
                f[i] = ninf;
                x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i0 + i < parts) {
                    f[i] = __ldcg(ml + at).x;
                    x[i] = __ldcg(reinterpret_cast<const float4*>(po + static_cast<int64_t>(at) * p.D + d));
                }
            }
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                const float a = fast_exp2(f[i] - use);
                o.x = fmaf(x[i].x, a, o.x);
                o.y = fmaf(x[i].y, a, o.y);
                o.z = fmaf(x[i].z, a, o.z);
                o.w = fmaf(x[i].w, a, o.w);
            }
        }
        const int qi = pc.tile * M + m;
        T* to = static_cast<T*>(p.out) + ((static_cast<int64_t>(pc.r.row0) + qi / p.G) * p.Hq + pc.h * p.G + qi % p.G) * p.D;
        store_four(to + d, l != 0.f ? make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f));
    }
}

}  // namespace attn
}  // namespace dspark
