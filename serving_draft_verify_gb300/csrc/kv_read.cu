// dspark_read_kv: rows of the paged cache back as float32 or bf16, and the size of a cache's pages.
//
// out[i][head][:] = cache[slot[i]][head][:], a stored 8- or 4-bit value times its scales in float32,
// rounded once.
//
// Bound by memory, mostly by what is written.  A thread has one piece of eight elements of a row
// (key or value, head, place) and moves it for eight rows at a time, all loads before the first store;
// where the rows lie is found once a block.  131001 rows of 8 heads of 128 from 4 bits to bf16: 108 us for 689 MB
// (6.4 TB/s; with four rows at a time 124, with two 178, with sixteen 122); from 8 bits 123 (6.6 TB/s), from
// bf16 159 (6.7); 65000 rows from 4 bits to float32 120 (5.1).
#include "kv_store.cuh"
#include "launch.cuh"

namespace dspark {
namespace {

constexpr int kItems = 8;
constexpr int kThreads = 128;
constexpr int kMaxRows = 256;                   // of a block
constexpr int64_t kAlone = 256;                 // rows up to which one launch does, as in kv_write.cu

struct ReadArgs {
    int64_t rows, k_stride, v_stride, slots;    // strides in elements
    int heads, D, page, rows_per_block, parts;  // parts: 8-element pieces of one row of one tensor
    int lanes;                                  // threads of a row: a power of two, or all
    bool alone;                                 // no clearing came before
    const int64_t* slot;
    const float *k_scale, *v_scale;
    const void *kc, *vc;
    void *k, *v;
    StatusBlock* status;
    Page4 g;
};

// Eight stored elements, and how they become floats.
template <int kCache>
struct Stored;
template <>
struct Stored<DSPARK_F32> : Eight<float> {
    __device__ void get(const uint8_t* p, const uint8_t*) { load(p); }
    __device__ void values(float* f, float) const { floats(f); }
};
template <>
struct Stored<DSPARK_BF16> : Eight<__nv_bfloat16> {
    __device__ void get(const uint8_t* p, const uint8_t*) { load(p); }
    __device__ void values(float* f, float) const { floats(f); }
};
template <>
struct Stored<DSPARK_E4M3> {
    uint2 w;
    __device__ void get(const uint8_t* p, const uint8_t*) { w = __ldg(reinterpret_cast<const uint2*>(p)); }
    __device__ void values(float* f, float scale) const {
        const uint32_t h[4] = {e4m3x2_f16x2(w.x), e4m3x2_f16x2(w.x >> 16), e4m3x2_f16x2(w.y), e4m3x2_f16x2(w.y >> 16)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = f16lo(h[i]) * scale;
            f[2 * i + 1] = f16hi(h[i]) * scale;
        }
    }
};
template <>
struct Stored<DSPARK_E2M1> {
    uint32_t w, s;
    __device__ void get(const uint8_t* p, const uint8_t* scale) {
        w = __ldg(reinterpret_cast<const uint32_t*>(p));
        s = __ldg(scale);
    }
    __device__ void values(float* f, float scale) const {
        uint32_t h[4];
        e2m1x8_f16(w, h);
        const float sg = e4m3_float(s) * scale;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = f16lo(h[i]) * sg;
            f[2 * i + 1] = f16hi(h[i]) * sg;
        }
    }
};
__device__ __forceinline__ void put_eight(float* to, const float* f) {
    reinterpret_cast<float4*>(to)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(to)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void put_eight(__nv_bfloat16* to, const float* f) {
    __nv_bfloat162 two[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) two[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(two);
}

template <typename T, int kCache>
__global__ void __launch_bounds__(kThreads) read_kv(const __grid_constant__ ReadArgs p) {
    // bytes to a row of head 0, and to its scales; -1: none
    __shared__ longlong2 s_from[kMaxRows];
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_block;
    const int64_t left = p.rows - row0;
    const int n = left < p.rows_per_block ? static_cast<int>(left) : p.rows_per_block;
    // Alone, the first block clears the status and looks at the slots of all rows.
    const bool all = p.alone && blockIdx.x == 0;
    if (all && threadIdx.x < 4) reinterpret_cast<uint32_t*>(p.status)[threadIdx.x] = 0;
    bool past = false;
    constexpr int kBits = kCache == DSPARK_E2M1 ? 4 : kCache == DSPARK_E4M3 ? 8 : kCache == DSPARK_BF16 ? 16 : 32;
    const int row_bytes = p.D * kBits / 8;
    const int64_t page_bytes = kCache == DSPARK_E2M1 ? p.g.whole : static_cast<int64_t>(p.page) * row_bytes;
    for (int r = threadIdx.x; r < (all ? static_cast<int>(p.rows) : n); r += kThreads) {
        const int64_t slot = p.slot[row0 + r];
        longlong2 from = make_longlong2(-1, -1);
        if (slot >= p.slots) {
            past = true;
        } else if (slot >= 0) {
            const int64_t block = (slot >> 32) == 0 ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.page) : slot / p.page;
            const int in = static_cast<int>(slot - block * p.page);
            from.x = block * p.heads * page_bytes + static_cast<int64_t>(in) * row_bytes;
            from.y = block * p.heads * page_bytes + p.g.codes + static_cast<int64_t>(in) * p.g.scale;
        }
        if (r < n) s_from[r] = from;
    }
    __syncthreads();
    if (past && (all || !p.alone)) tell(p.status, DSPARK_ERR_DEVICE_CHECK, 1);
    const int groups = kThreads / p.lanes, mine = threadIdx.x / p.lanes, per_head = p.D / 8;
    for (int e = threadIdx.x % p.lanes; e < 2 * p.parts; e += p.lanes) {
        const bool is_v = e >= p.parts;
        const int part = is_v ? e - p.parts : e, head = part / per_head, at = (part - head * per_head) * 8;
        const int64_t stride = is_v ? p.v_stride : p.k_stride;
        T* out = static_cast<T*>(is_v ? p.v : p.k) + (row0 + mine) * stride + static_cast<int64_t>(part) * 8;
        const uint8_t* cache = static_cast<const uint8_t*>(is_v ? p.vc : p.kc) + head * page_bytes;
        const uint8_t *code = cache + at * kBits / 8, *scales = cache + at / 16;
        const float scale = kBits <= 8 ? __ldg((is_v ? p.v_scale : p.k_scale) + head) : 1.f;
        for (int r = mine; r < n; r += kItems * groups, out += kItems * groups * stride) {
            Stored<kCache> x[kItems];
            bool real[kItems];
#pragma unroll
            for (int j = 0; j < kItems; ++j) {
                longlong2 from = make_longlong2(-1, -1);
                if (r + j * groups < n) {
                    if constexpr (kBits == 4) from = s_from[r + j * groups];
                    else from.x = s_from[r + j * groups].x;
                }
                real[j] = from.x >= 0;
                if (real[j]) x[j].get(code + from.x, scales + from.y);
            }
#pragma unroll
            for (int j = 0; j < kItems; ++j) {
                if (!real[j]) continue;
                float f[8];
                x[j].values(f, scale);
                put_eight(out + j * groups * stride, f);
            }
        }
    }
    if (blockIdx.x == 0) head_cleared();
}

template <typename T>
void (*kernel_of(dspark_dtype_t c))(ReadArgs) {
    switch (c) {
        case DSPARK_F32: return read_kv<T, DSPARK_F32>;
        case DSPARK_BF16: return read_kv<T, DSPARK_BF16>;
        case DSPARK_E4M3: return read_kv<T, DSPARK_E4M3>;
        default: return read_kv<T, DSPARK_E2M1>;
    }
}

}  // namespace
}  // namespace dspark

extern "C" size_t dspark_kv_page_bytes(int page, int D, dspark_dtype_t cache_dt) {
    using namespace dspark;
    if (page < 1 || D < 8 || D > 256 || D % 8 != 0 || cache_dt < DSPARK_F32 || cache_dt > DSPARK_E2M1) return 0;
    const size_t n = static_cast<size_t>(page) * D;
    if (cache_dt != DSPARK_E2M1) return n * (cache_dt == DSPARK_F32 ? 4 : cache_dt == DSPARK_BF16 ? 2 : 1);
    return D % 32 != 0 || n > 0x7fffffffll - 1024 ? 0 : static_cast<size_t>(page4_of(page, D).whole);
}

extern "C" size_t dspark_read_kv_workspace_size(void) { return dspark::kStatusBytes; }

extern "C" dspark_status_t dspark_read_kv(int64_t rows, int Hkv, int D, int page, int num_blocks, dspark_dtype_t dt,
                                          dspark_dtype_t cache_dt, const int64_t* slot, const void* k_cache,
                                          const void* v_cache, const float* k_scale, const float* v_scale, void* k,
                                          int64_t k_stride, void* v, int64_t v_stride, void* workspace,
                                          size_t workspace_bytes, dspark_stream_t stream) {
    using namespace dspark;
    const bool scaled = cache_dt == DSPARK_E4M3 || cache_dt == DSPARK_E2M1;
    if (rows < 0 || rows > 0x7fffffffll || Hkv < 1 || Hkv > 1024 || D < 8 || D > 256 || D % 8 != 0 || page < 1 ||
        num_blocks < 1)
        return DSPARK_ERR_INVALID_ARGUMENT;
    if ((dt != DSPARK_BF16 && dt != DSPARK_F32) || (!scaled && cache_dt != DSPARK_BF16 && cache_dt != DSPARK_F32))
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (scaled && (D % (cache_dt == DSPARK_E4M3 ? 16 : 32) != 0 || k_scale == nullptr || v_scale == nullptr))
        return DSPARK_ERR_INVALID_ARGUMENT;
    const int64_t width = static_cast<int64_t>(Hkv) * D, align = dt == DSPARK_BF16 ? 8 : 4;
    if (k_stride < width || v_stride < width || k_stride % align != 0 || v_stride % align != 0)
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (k_cache == nullptr || v_cache == nullptr || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k) ||
        !aligned16(v) || (rows > 0 && (k == nullptr || v == nullptr || slot == nullptr)))
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (cache_dt == DSPARK_E2M1 && static_cast<int64_t>(page) * D > 0x7fffffffll - 1024) return DSPARK_ERR_UNSUPPORTED;
    if (workspace == nullptr || !aligned256(workspace)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < dspark_read_kv_workspace_size()) return DSPARK_ERR_WORKSPACE_TOO_SMALL;
    clear_stale_error();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) return clear_status(workspace, s);
    ReadArgs p{};
    p.rows = rows, p.k_stride = k_stride, p.v_stride = v_stride;
    p.slots = static_cast<int64_t>(num_blocks) * page;
    p.heads = Hkv, p.D = D, p.page = page, p.g = page4_of(page, D);
    p.parts = static_cast<int>(width / 8);
    // Eight rows a thread, and fewer where the rows would not fill the GPU.
    p.lanes = 1;
    while (p.lanes < kThreads && p.lanes < 2 * p.parts) p.lanes *= 2;
    const int groups = kThreads / p.lanes;
    p.rows_per_block = groups * kItems < kMaxRows ? groups * kItems : kMaxRows;
    while (p.rows_per_block > 1 && (rows + p.rows_per_block - 1) / p.rows_per_block < 2 * sm_count(current_device()))
        p.rows_per_block /= 2;
    p.alone = rows <= kAlone;
    p.slot = slot, p.k_scale = k_scale, p.v_scale = v_scale, p.kc = k_cache, p.vc = v_cache, p.k = k, p.v = v;
    p.status = static_cast<StatusBlock*>(workspace);
    const unsigned grid = static_cast<unsigned>((rows + p.rows_per_block - 1) / p.rows_per_block);
    void (*kernel)(ReadArgs) = dt == DSPARK_BF16 ? kernel_of<__nv_bfloat16>(cache_dt) : kernel_of<float>(cache_dt);
    if (p.alone) {
        kernel<<<grid, kThreads, 0, s>>>(p);
        return launch_status();
    }
    return launch_cleared(workspace, kStatusBytes, kernel, dim3(grid), kThreads, 0, s, p);
}
