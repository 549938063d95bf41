// dspark_paged_attention: attention of a step's rows over the paged cache.
// attn.cuh has the mathematics, the division of the work and the joining.
#include <cuda_fp8.h>

#include <type_traits>

#include "attn.cuh"
#include "attn_mma.cuh"
#include "attn_tc.cuh"

namespace dspark {
namespace attn {
namespace {

// Query rows of a key head above which tcgen05 takes over, by max_rows.  32 heads on 8, us on the
// warp-level instructions and on tcgen05: 64 requests of up to 4000 keys, 12 rows a request (48 query
// rows) 188 and 205, 16 rows 229 and 222, 17 rows 284 and 240; 128 requests of up to 6000 keys, 17 rows
// 723 and 501.  Short caches favour the former longer (256 requests of up to 500 keys, 16 rows: 242 and
// 302), and so do steps whose requests have far fewer rows than max_rows (64 requests of one row, up to
// 16384 keys: 371 and, called with max_rows 17, 629), but lengths and rows are on the device.
constexpr int kWide = 64;

// ------------------------------------------------------------ float32 rows ---
// Sixteen query rows (up to four a warp) over 32 keys a unit, float32 throughout: a lane is a key
// for the scores and has pairs of columns of the values.  The next unit's keys and values are copied
// (asynchronously, as they are stored) while this one's are computed on.
constexpr int kSimtM = 16, kSimtKT = 32, kSimtThreads = 128;

// Four adjacent stored elements, and two, as float.
template <typename C>
__device__ __forceinline__ float4 four_of(const unsigned char* at);
template <>
__device__ __forceinline__ float4 four_of<float>(const unsigned char* at) {
    return *reinterpret_cast<const float4*>(at);
}
template <>
__device__ __forceinline__ float4 four_of<__nv_fp8_e4m3>(const unsigned char* at) {
    return static_cast<float4>(*reinterpret_cast<const __nv_fp8x4_e4m3*>(at));
}
template <typename C>
__device__ __forceinline__ float2 two_of(const unsigned char* row, int d);
template <>
__device__ __forceinline__ float2 two_of<float>(const unsigned char* row, int d) {
    return *reinterpret_cast<const float2*>(row + 4 * d);
}
template <>
__device__ __forceinline__ float2 two_of<__nv_fp8_e4m3>(const unsigned char* row, int d) {
    return static_cast<float2>(*reinterpret_cast<const __nv_fp8x2_e4m3*>(row + d));
}
template <typename C>
constexpr int simt_row(int D) {                    // bytes of a staged row
    return D * static_cast<int>(sizeof(C)) + 16;
}
template <typename C>
constexpr size_t simt_smem(int D) {
    return 4 * static_cast<size_t>(kSimtKT) * simt_row<C>(D) + (static_cast<size_t>(kSimtM) * D + kSimtM * kSimtKT) * 4;
}

template <typename C, int kCols>
__global__ void __launch_bounds__(kSimtThreads) attend_simt(const __grid_constant__ Args p) {
    constexpr int M = kSimtM, KT = kSimtKT;
    extern __shared__ float4 smem4[];
    const int row_bytes = simt_row<C>(p.D), chunks = p.D * static_cast<int>(sizeof(C)) / 16;
    unsigned char* s_kv = reinterpret_cast<unsigned char*>(smem4);                  // [2 stages][keys, values][KT] rows
    float* s_q = reinterpret_cast<float*>(s_kv + 4 * KT * row_bytes);              // [M][D]
    float* s_p = s_q + M * p.D;                        // [M][KT]: exp of the scores, -1 where masked
    __shared__ long long scratch[38];
    __shared__ float2 s_row[M];
    __shared__ int s_flag;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const float ninf = -__uint_as_float(0x7f800000u);

    const Start st = find_start<M, KT, kSimtThreads>(p, scratch);
    Walk<M, KT> walk(p, st);
    Piece pc;
    while (walk.next(pc)) {
        const int left = pc.r.n * p.G - pc.tile * M, valid = left < M ? left : M;
        // lane j has the place (in rows) of key j of a unit, found a unit ahead of its copy
        auto find_rows = [&](int u) -> int64_t {
            const int key = pc.span.lo + u * KT + lane;
            if (u >= pc.u1 || key < pc.span.seen || key >= pc.span.hi) return 0;
            const int blk = key / p.page;
            return (static_cast<int64_t>(page_id(p, pc.b, blk)) * p.Hkv + pc.h) * p.page + (key - blk * p.page);
        };
        auto load = [&](int u, int64_t rows) {
            if (u < pc.u1) {
                const uint32_t to = smem_u32(s_kv) + ((u - pc.u0) & 1) * 2 * KT * row_bytes;
                const int n = KT * chunks;             // a multiple of the warp's 32
                for (int e = tid; e < n; e += kSimtThreads) {
                    const int r = e / chunks, c = e - r * chunks;
                    const int64_t row = __shfl_sync(0xffffffffu, rows, r);
                    const int key = pc.span.lo + u * KT + r;
                    const bool real = key >= pc.span.seen && key < pc.span.hi;
                    const int64_t at = real ? row * (p.D * static_cast<int>(sizeof(C))) + c * 16 : 0;
                    copy16(to + r * row_bytes + c * 16, static_cast<const char*>(p.kc) + at, real);
                    copy16(to + (KT + r) * row_bytes + c * 16, static_cast<const char*>(p.vc) + at, real);
                }
            }
            copy_commit();
        };
        __syncthreads();                               // the last piece is done with the stages
        load(pc.u0, find_rows(pc.u0));
        int64_t rows = find_rows(pc.u0 + 1);
        const float qs = p.scale_log2 * (p.k_scale != nullptr ? p.k_scale[pc.h] : 1.f);
        for (int e = tid; e < M * p.D / 4; e += kSimtThreads) {
            const int m = e / (p.D / 4), d = (e - m * (p.D / 4)) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (m < valid) {
                const int qi = pc.tile * M + m;
                x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.q) +
                                                          (static_cast<int64_t>(pc.r.row0) + qi / p.G) * p.q_stride +
                                                          static_cast<int64_t>(pc.h * p.G + qi % p.G) * p.D + d));
            }
            *reinterpret_cast<float4*>(s_q + m * p.D + d) = make_float4(x.x * qs, x.y * qs, x.z * qs, x.w * qs);
        }
        float mx[4], l[4], o[4][kCols];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            mx[r] = ninf;
            l[r] = 0.f;
#pragma unroll
            for (int c = 0; c < kCols; ++c) o[r][c] = 0.f;
        }
        for (int u = pc.u0; u < pc.u1; ++u) {
            const int k0 = pc.span.lo + u * KT;
            load(u + 1, rows);
            rows = find_rows(u + 2);
            copy_wait<1>();
            __syncthreads();
            const unsigned char* s_k = s_kv + ((u - pc.u0) & 1) * 2 * KT * row_bytes;
            const unsigned char* s_v = s_k + KT * row_bytes;
            // The warp's rows are w, w + 4, ...: a tile with few rows has them spread over the warps.
            auto compute = [&](auto count) {
                constexpr int R = decltype(count)::value;
                float s[R] = {};
#pragma unroll 4
                for (int d = 0; d < p.D; d += 4) {
                    const float4 k = four_of<C>(s_k + lane * row_bytes + d * sizeof(C));
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float4 q = *reinterpret_cast<const float4*>(s_q + (w + 4 * r) * p.D + d);
                        s[r] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[r]))));
                    }
                }
                bool masked = false;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int m = w + 4 * r, pos = pc.r.len + (pc.tile * M + m) / p.G, key = k0 + lane;
                    const bool seen = m < valid && key <= pos && (p.window == 0 || key > pos - p.window);
                    masked |= !seen;
                    const float nm = fmaxf(mx[r], warp_max(seen ? s[r] : ninf));
                    const float use = nm == ninf ? 0.f : nm;
                    const float a = fast_exp2(mx[r] - use), e = seen ? fast_exp2(s[r] - use) : 0.f;
                    mx[r] = nm;
                    l[r] = l[r] * a + e;               // this lane's keys; the lanes' sums meet at the end
#pragma unroll
                    for (int c = 0; c < kCols; ++c) o[r][c] *= a;
                    s_p[m * KT + lane] = seen ? e : -1.f;
                }
                // Four keys at a time.  A masked key's value stays out even where it is not a number; only
                // units with masked keys ask.
                masked = __any_sync(0xffffffffu, masked);
                __syncwarp();
#pragma unroll 1
                for (int j = 0; j < KT; j += 4) {
                    float4 e[R];
#pragma unroll
                    for (int r = 0; r < R; ++r) e[r] = *reinterpret_cast<const float4*>(s_p + (w + 4 * r) * KT + j);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float2 v[kCols / 2];
#pragma unroll
                        for (int c = 0; c < kCols / 2; ++c)
                            v[c] = 2 * lane + 64 * c < p.D ? two_of<C>(s_v + (j + i) * row_bytes, 2 * lane + 64 * c) : make_float2(0.f, 0.f);
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const float x = i == 0 ? e[r].x : i == 1 ? e[r].y : i == 2 ? e[r].z : e[r].w;
                            if (!masked || !(x < 0.f)) {
#pragma unroll
                                for (int c = 0; c < kCols / 2; ++c) {
                                    o[r][2 * c] = fmaf(x, v[c].x, o[r][2 * c]);
                                    o[r][2 * c + 1] = fmaf(x, v[c].y, o[r][2 * c + 1]);
                                }
                            }
                        }
                    }
                }
            };
            const int rows_of_warp = (valid - w + 3) / 4;
            if (rows_of_warp > 2) compute(std::integral_constant<int, 4>{});
            else if (rows_of_warp == 2) compute(std::integral_constant<int, 2>{});
            else if (rows_of_warp == 1) compute(std::integral_constant<int, 1>{});
            __syncthreads();
        }
        copy_wait<0>();
        const float vs = p.v_scale != nullptr ? p.v_scale[pc.h] : 1.f;
        const bool whole = pc.whole();
        const int64_t place = part_place(blockIdx.x, pc.u0 == 0) * M;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int m = w + 4 * r;
            if (m >= valid) continue;
            l[r] = warp_sum(l[r]);
            const int qi = pc.tile * M + m, head = pc.h * p.G + qi % p.G;
            const int64_t row = static_cast<int64_t>(pc.r.row0) + qi / p.G, at = place + m;
            float* to = whole ? static_cast<float*>(p.out) + (row * p.Hq + head) * p.D : p.part_o + at * p.D;
            const float f = !whole ? vs : l[r] != 0.f ? vs / l[r] : 0.f;
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c)
                if (2 * lane + 64 * c < p.D)
                    *reinterpret_cast<float2*>(to + 2 * lane + 64 * c) =
                        whole && l[r] == 0.f ? make_float2(0.f, 0.f) : make_float2(o[r][2 * c] * f, o[r][2 * c + 1] * f);
            if (lane == 0) {
                if (!whole) reinterpret_cast<float2*>(p.part_ml)[at] = make_float2(mx[r], l[r]);
                else if (p.lse != nullptr) p.lse[row * p.Hq + head] = lse_of(mx[r], l[r]);
            }
        }
        if (!whole && part_done(p, pc, st, &s_flag, tid, [] { __syncthreads(); }))
            join_parts<float, M, kSimtThreads>(p, pc, st, s_row, tid, [] { __syncthreads(); });
    }
    if (blockIdx.x == 0) head_cleared();
}

template <typename C, int kCols>
dspark_status_t launch_simt(const Args& p, cudaStream_t s) {
    static OncePerDevice once;
    if (once.run(current_device(), [] {
            return cudaFuncSetAttribute(attend_simt<C, kCols>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(simt_smem<C>(32 * kCols)));
        }) != cudaSuccess)
        return DSPARK_ERR_CUDA;
    const size_t smem = simt_smem<C>(p.D);
    const int per_sm = smem <= 52 * 1024 ? 4 : smem <= 108 * 1024 ? 2 : 1;
    const int grid = grid_for(sm_count(current_device()) * per_sm, kSimtM);
    if (grid < 1) return DSPARK_ERR_CUDA;
    return launch_cleared(p.status, kHeadBytes, attend_simt<C, kCols>, dim3(grid), kSimtThreads, smem, s, p);
}
template <typename C>
dspark_status_t launch_f32(const Args& p, cudaStream_t s) {
    if (p.D <= 64) return launch_simt<C, 2>(p, s);
    if (p.D <= 128) return launch_simt<C, 4>(p, s);
    return launch_simt<C, 8>(p, s);
}

// bf16 rows: sixteen query rows at a time on the warp-level instructions, or 128 on tcgen05 where a
// request may have more rows than kWide.
template <bool kFp8>
dspark_status_t launch_bf16(const Args& p, cudaStream_t s) {
    if constexpr (!kFp8)
        if (static_cast<int64_t>(p.max_rows) * p.G > kWide && tc_fits(p)) return p.D <= 64 ? launch_tc<64>(p, s) : launch_tc<128>(p, s);
    if (p.D <= 64) return launch_mma<kFp8, 64>(p, s);
    if (p.D <= 128) return launch_mma<kFp8, 128>(p, s);
    return launch_mma<kFp8, 256>(p, s);
}

}  // namespace
}  // namespace attn
}  // namespace dspark

extern "C" size_t dspark_paged_attention_workspace_size(int D) {
    using namespace dspark;
    if (D < 1) return 0;
    return kStatusBytes + attn::kCounterBytes + static_cast<size_t>(attn::kMaxPartRows) * (D + 2) * 4;
}

extern "C" dspark_status_t dspark_paged_attention(
    int B, int64_t rows, int max_rows, int Hq, int Hkv, int D, int page, int max_blocks, int num_blocks,
    dspark_dtype_t dt, dspark_dtype_t cache_dt, const void* q, int64_t q_stride, const int32_t* row_offset,
    const int32_t* len, const int32_t* block_table, int64_t ld_table, const void* k_cache, const void* v_cache,
    const float* k_scale, const float* v_scale, float scale, int window, void* out, float* lse, void* workspace,
    size_t workspace_bytes, dspark_stream_t stream) {
    using namespace dspark;
    if (B < 1 || B > 65535 || rows < 0 || rows > 0x7fffffffll || max_rows < (rows > 0 ? 1 : 0) || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 ||
        Hq > 1024 || D < 8 || D > 256 || D % 8 != 0 || page < 1 || max_blocks < 1 || num_blocks < 1 ||
        ld_table < max_blocks || window < 0)
        return DSPARK_ERR_INVALID_ARGUMENT;
    if ((dt != DSPARK_BF16 && dt != DSPARK_F32) || (cache_dt != dt && cache_dt != DSPARK_E4M3))
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (cache_dt == DSPARK_E4M3 && (D % 16 != 0 || k_scale == nullptr || v_scale == nullptr))
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (!(scale == scale) || scale - scale != 0.f) return DSPARK_ERR_INVALID_ARGUMENT;
    const int64_t align = dt == DSPARK_BF16 ? 8 : 4;
    if (q_stride < static_cast<int64_t>(Hq) * D || q_stride % align != 0) return DSPARK_ERR_INVALID_ARGUMENT;
    if (row_offset == nullptr || len == nullptr || block_table == nullptr || k_cache == nullptr || v_cache == nullptr ||
        (rows > 0 && (q == nullptr || out == nullptr)) || !aligned16(q) || !aligned16(out) || !aligned16(k_cache) ||
        !aligned16(v_cache))
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (static_cast<int64_t>(max_blocks) * page > 0x7fffffffll - 1024 ||
        static_cast<int64_t>(max_rows) * (Hq / Hkv) > 0x7fffffffll - 1024)
        return DSPARK_ERR_UNSUPPORTED;
    if (workspace == nullptr || !aligned256(workspace)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < dspark_paged_attention_workspace_size(D)) return DSPARK_ERR_WORKSPACE_TOO_SMALL;
    clear_stale_error();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) return clear_status(workspace, s);
    attn::Args p{};
    p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.G = Hq / Hkv, p.D = D, p.page = page, p.max_blocks = max_blocks;
    p.num_blocks = num_blocks, p.max_rows = max_rows, p.window = window, p.rows = rows, p.ld_table = ld_table;
    p.q_stride = q_stride, p.q = q, p.row_offset = row_offset, p.length = len, p.table = block_table;
    p.kc = k_cache, p.vc = v_cache;
    if (cache_dt == DSPARK_E4M3) p.k_scale = k_scale, p.v_scale = v_scale;
    p.scale_log2 = scale * kLog2e, p.out = out, p.lse = lse;
    char* ws = static_cast<char*>(workspace);
    p.status = reinterpret_cast<StatusBlock*>(ws);
    p.counters = reinterpret_cast<uint32_t*>(ws + kStatusBytes);
    p.part_ml = reinterpret_cast<float*>(ws + kStatusBytes + attn::kCounterBytes);
    p.part_o = p.part_ml + 2 * static_cast<size_t>(attn::kMaxPartRows);
    const bool fp8 = cache_dt == DSPARK_E4M3;
    if (dt == DSPARK_BF16) return fp8 ? attn::launch_bf16<true>(p, s) : attn::launch_bf16<false>(p, s);
    return fp8 ? attn::launch_f32<__nv_fp8_e4m3>(p, s) : attn::launch_f32<float>(p, s);
}
