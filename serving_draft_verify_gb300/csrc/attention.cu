// dspark_paged_attention: attention of a step's rows over the paged cache.
// attn.cuh has the mathematics, the division of the work and the joining.
#include <cuda_fp8.h>

#include "attn.cuh"
#include "attn_mma.cuh"
#include "attn_tc.cuh"

namespace dspark {
namespace attn {
namespace {

// ------------------------------------------------------------ float32 rows ---
// Sixteen query rows (four a warp) over 32 keys a unit, float32 throughout: a lane is
// a key for the scores and a column for the values.
constexpr int kSimtM = 16, kSimtKT = 32, kSimtThreads = 128;

template <typename T>
__device__ __forceinline__ float4 load4(const void* base, int64_t i);
template <>
__device__ __forceinline__ float4 load4<float>(const void* base, int64_t i) {
    return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + i));
}
template <>
__device__ __forceinline__ float4 load4<__nv_fp8_e4m3>(const void* base, int64_t i) {
    const __nv_fp8x4_e4m3 u = *reinterpret_cast<const __nv_fp8x4_e4m3*>(static_cast<const uint8_t*>(base) + i);
    return static_cast<float4>(u);
}

template <typename C, int kCols>
__global__ void __launch_bounds__(kSimtThreads) attend_simt(const __grid_constant__ Args p) {
    constexpr int M = kSimtM, KT = kSimtKT;
    extern __shared__ float4 smem4[];
    const int ld = p.D + 4;
    float* s_q = reinterpret_cast<float*>(smem4);      // [M][D]
    float* s_k = s_q + M * p.D;                        // [KT][ld]
    float* s_v = s_k + KT * ld;                        // [KT][ld]
    float* s_p = s_v + KT * ld;                        // [M][KT]: exp of the scores, -1 where masked
    __shared__ long long scratch[34];
    __shared__ float2 s_row[M];
    __shared__ int s_flag;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const float ninf = -__uint_as_float(0x7f800000u);

    const Start st = find_start<M, KT, kSimtThreads>(p, scratch);
    Walk<M, KT> walk(p, st);
    Piece pc;
    while (walk.next(pc)) {
        __syncthreads();
        const int valid = static_cast<int>(min(static_cast<int64_t>(M), static_cast<int64_t>(pc.r.n) * p.G - static_cast<int64_t>(pc.tile) * M));
        const float qs = p.scale_log2 * (p.k_scale != nullptr ? p.k_scale[pc.h] : 1.f);
        for (int e = tid; e < M * p.D / 4; e += kSimtThreads) {
            const int m = e / (p.D / 4), d = (e - m * (p.D / 4)) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (m < valid) {
                const int qi = pc.tile * M + m;
                x = load4<float>(p.q, (static_cast<int64_t>(pc.r.row0) + qi / p.G) * p.q_stride +
                                      static_cast<int64_t>(pc.h * p.G + qi % p.G) * p.D + d);
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
            __syncthreads();
            for (int e = tid; e < KT * p.D / 4; e += kSimtThreads) {
                const int j = e / (p.D / 4), d = (e - j * (p.D / 4)) * 4, key = k0 + j;
                float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
                if (key < pc.span.hi) {
                    const int blk = key / p.page;
                    const int64_t at =
                        ((static_cast<int64_t>(page_id(p, pc.b, blk)) * p.Hkv + pc.h) * p.page + (key - blk * p.page)) * p.D + d;
                    k = load4<C>(p.kc, at);
                    v = load4<C>(p.vc, at);
                }
                *reinterpret_cast<float4*>(s_k + j * ld + d) = k;
                *reinterpret_cast<float4*>(s_v + j * ld + d) = v;
            }
            __syncthreads();
            float s[4] = {0.f, 0.f, 0.f, 0.f};
            for (int d = 0; d < p.D; d += 4) {
                const float4 k = *reinterpret_cast<const float4*>(s_k + lane * ld + d);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float4 q = *reinterpret_cast<const float4*>(s_q + (4 * w + r) * p.D + d);
                    s[r] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[r]))));
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int m = 4 * w + r, pos = pc.r.len + (pc.tile * M + m) / p.G, key = k0 + lane;
                const bool seen = m < valid && key <= pos && (p.window == 0 || key > pos - p.window);
                const float nm = fmaxf(mx[r], warp_max(seen ? s[r] : ninf));
                const float use = nm == ninf ? 0.f : nm;
                const float a = fast_exp2(mx[r] - use), e = seen ? fast_exp2(s[r] - use) : 0.f;
                mx[r] = nm;
                l[r] = l[r] * a + warp_sum(e);
#pragma unroll
                for (int c = 0; c < kCols; ++c) o[r][c] *= a;
                s_p[m * KT + lane] = seen ? e : -1.f;
            }
            __syncwarp();
            for (int j = 0; j < KT; ++j) {
                float v[kCols];
#pragma unroll
                for (int c = 0; c < kCols; ++c) v[c] = lane + 32 * c < p.D ? s_v[j * ld + lane + 32 * c] : 0.f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float e = s_p[(4 * w + r) * KT + j];
                    // a masked key's value stays out even where it is not a number
                    if (!(e < 0.f)) {
#pragma unroll
                        for (int c = 0; c < kCols; ++c) o[r][c] = fmaf(e, v[c], o[r][c]);
                    }
                }
            }
        }
        const float vs = p.v_scale != nullptr ? p.v_scale[pc.h] : 1.f;
        if (pc.whole()) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int m = 4 * w + r;
                if (m >= valid) continue;
                const int qi = pc.tile * M + m, head = pc.h * p.G + qi % p.G;
                const int64_t row = static_cast<int64_t>(pc.r.row0) + qi / p.G;
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    if (lane + 32 * c < p.D)
                        static_cast<float*>(p.out)[(row * p.Hq + head) * p.D + lane + 32 * c] = l[r] != 0.f ? o[r][c] * vs / l[r] : 0.f;
                if (lane == 0 && p.lse != nullptr) p.lse[row * p.Hq + head] = lse_of(mx[r], l[r]);
            }
        } else {
            const int64_t place = part_place(blockIdx.x, pc.u0 == 0) * M;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t at = place + 4 * w + r;
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    if (lane + 32 * c < p.D) p.part_o[at * p.D + lane + 32 * c] = o[r][c] * vs;
                if (lane == 0) reinterpret_cast<float2*>(p.part_ml)[at] = make_float2(mx[r], l[r]);
            }
            if (part_done(p, pc, st, &s_flag, tid, [] { __syncthreads(); })) join_parts<float, M, kSimtThreads>(p, pc, st, s_row, tid, [] { __syncthreads(); });
        }
    }
}

template <typename C, int kCols>
dspark_status_t launch_simt(const Args& p, cudaStream_t s) {
    const size_t smem = (static_cast<size_t>(kSimtM) * p.D + 2 * kSimtKT * (p.D + 4) + kSimtM * kSimtKT) * 4;
    static OncePerDevice once;
    if (once.run(current_device(), [] {
            return cudaFuncSetAttribute(attend_simt<C, kCols>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (kSimtM * 256 + 2 * kSimtKT * 260 + kSimtM * kSimtKT) * 4);
        }) != cudaSuccess)
        return DSPARK_ERR_CUDA;
    const int grid = grid_for(sm_count(current_device()) * (kCols <= 4 ? 4 : 2), kSimtM);
    if (grid < 1) return DSPARK_ERR_CUDA;
    attend_simt<C, kCols><<<grid, kSimtThreads, smem, s>>>(p);
    return launch_status();
}
template <typename C>
dspark_status_t launch_f32(const Args& p, cudaStream_t s) {
    if (p.D <= 64) return launch_simt<C, 2>(p, s);
    if (p.D <= 128) return launch_simt<C, 4>(p, s);
    return launch_simt<C, 8>(p, s);
}

// bf16 rows: the instructions take 16 query rows at a time, two such tiles where a request has
// more than 16 (and the output rows still fit the registers).
template <bool kFp8>
dspark_status_t launch_bf16(const Args& p, cudaStream_t s) {
    const int64_t most = static_cast<int64_t>(p.max_rows) * p.G;
    if constexpr (!kFp8)
        if (most > 32 && tc_fits(p)) return p.D <= 64 ? launch_tc<64>(p, s) : launch_tc<128>(p, s);
    const bool two = most > 16;
    if (p.D <= 64) return two ? launch_mma<kFp8, 2, 64>(p, s) : launch_mma<kFp8, 1, 64>(p, s);
    if (p.D <= 128) return two ? launch_mma<kFp8, 2, 128>(p, s) : launch_mma<kFp8, 1, 128>(p, s);
    return launch_mma<kFp8, 1, 256>(p, s);
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
    if (B < 1 || B > 65535 || rows < 0 || rows > 0x7fffffffll || max_rows < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 ||
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
    if (cudaMemsetAsync(workspace, 0, kStatusBytes + attn::kCounterBytes, s) != cudaSuccess) return DSPARK_ERR_CUDA;
    if (rows == 0) return DSPARK_OK;
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
