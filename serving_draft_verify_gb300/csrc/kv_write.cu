// dspark_write_kv: the keys and values of a step's rows into the paged cache.
//
// cache[slot / page][head][slot % page][:] = row[head][:], copied, or stored in
// 8 bits as e4m3(clamp(x / scale[head], +-448)), rounded to nearest even.  The
// quotient is formed in float32 by an IEEE division; NaN stays NaN.  4-bit caches are
// written by the kernel of rotate.cu, without a rotation.
//
// Bound by memory: each element is read once and written once.  A thread has one piece of eight
// elements of a row (key or value, head, place) and moves it for four rows at a time, all loads
// before the first store, so that the arithmetic of places is done once a thread and once a row.
// 16384 rows of 8 heads of 128: bf16 24 us (134 MB, 5.6 TB/s), to 8 bits 25 us (100 MB); with two
// rows at a time 37 and 33 us, with eight 24 and 27, with blocks of 256 threads 28 to 8 bits.
// float32 47 us (268 MB, 5.7 TB/s), to 8 bits 39 us (168 MB), caches flushed before each.
#include "launch.cuh"
#include "rotate.cuh"

namespace dspark {
namespace {

constexpr int kItems = 4;
constexpr int kThreads = 128;
constexpr int kMaxRows = 256;                   // of a block
// Rows up to which a call is one launch: its first block clears the status and looks at all slots
// instead of a clearing launch and every block at its own.  us in a graph so and with the clearing
// launch (8 heads of 128, bf16): 16 rows 2.2 and 2.9, 256 rows 2.7 and 3.1, 1024 rows 4.6 and 3.6.
constexpr int64_t kAlone = 256;

struct WriteArgs {
    int64_t rows, k_stride, v_stride, slots;    // strides in elements
    int heads, D, page, rows_per_block, parts;  // parts: 8-element pieces of one row of one tensor
    int lanes;                                  // threads of a row: a power of two, or all
    bool alone;                                 // no clearing came before
    const void *k, *v;
    const int64_t* slot;
    const float *k_scale, *v_scale;
    void *kc, *vc;
    StatusBlock* status;
};

template <typename T, bool kFp8>
__global__ void __launch_bounds__(kThreads) write_kv(WriteArgs p) {
    __shared__ int64_t s_to[kMaxRows];          // a row's first element of head 0 in the cache, -1: none
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_block;
    const int64_t left = p.rows - row0;
    const int n = left < p.rows_per_block ? static_cast<int>(left) : p.rows_per_block;
    // Alone, the first block clears the status and looks at the slots of all rows.
    const bool all = p.alone && blockIdx.x == 0;
    if (all && threadIdx.x < 4) reinterpret_cast<uint32_t*>(p.status)[threadIdx.x] = 0;
    bool past = false;
    for (int r = threadIdx.x; r < (all ? static_cast<int>(p.rows) : n); r += kThreads) {
        const int64_t slot = p.slot[row0 + r];
        int64_t to = -1;
        if (slot >= p.slots) {
            past = true;
        } else if (slot >= 0) {
            const int64_t block = (slot >> 32) == 0 ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.page) : slot / p.page;
            to = (block * p.heads * p.page + (slot - block * p.page)) * p.D;
        }
        if (r < n) s_to[r] = to;
    }
    __syncthreads();
    if (past && (all || !p.alone)) tell(p.status, DSPARK_ERR_DEVICE_CHECK, 1);
    const int groups = kThreads / p.lanes, mine = threadIdx.x / p.lanes, per_head = p.D / 8;
    for (int e = threadIdx.x % p.lanes; e < 2 * p.parts; e += p.lanes) {
        const bool is_v = e >= p.parts;
        const int part = is_v ? e - p.parts : e, head = part / per_head;
        const int64_t within = static_cast<int64_t>(head) * p.page * p.D + (part - head * per_head) * 8;
        const int64_t stride = is_v ? p.v_stride : p.k_stride;
        const T* from = static_cast<const T*>(is_v ? p.v : p.k) + row0 * stride + static_cast<int64_t>(part) * 8;
        void* cache = is_v ? p.vc : p.kc;
        const float scale = kFp8 ? __ldg((is_v ? p.v_scale : p.k_scale) + head) : 1.f, inv = kFp8 ? __fdiv_rn(1.f, scale) : 1.f;
        const float margin = margin_of(scale);
        for (int r0 = mine; r0 < n; r0 += kItems * groups) {
            Eight<T> x[kItems];
            int64_t to[kItems];
#pragma unroll
            for (int j = 0; j < kItems; ++j) {
                const int r = r0 + j * groups;
                to[j] = r < n ? s_to[r] : -1;
                if (to[j] >= 0) x[j].load(from + r * stride);
            }
#pragma unroll
            for (int j = 0; j < kItems; ++j) {
                if (to[j] < 0) continue;
                if constexpr (kFp8) {
                    float f[8];
                    x[j].floats(f);
                    uint32_t w[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        w[h] = stored(f[4 * h], f[4 * h + 1], scale, inv, margin) | (stored(f[4 * h + 2], f[4 * h + 3], scale, inv, margin) << 16);
                    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + to[j] + within) = make_uint2(w[0], w[1]);
                } else {
                    x[j].store(static_cast<T*>(cache) + to[j] + within);
                }
            }
        }
    }
    if (blockIdx.x == 0) head_cleared();
}

}  // namespace
}  // namespace dspark

extern "C" size_t dspark_write_kv_workspace_size(void) { return dspark::kStatusBytes; }

extern "C" dspark_status_t dspark_write_kv(int64_t rows, int Hkv, int D, int page, int num_blocks, dspark_dtype_t dt,
                                           dspark_dtype_t cache_dt, const void* k, int64_t k_stride, const void* v,
                                           int64_t v_stride, const int64_t* slot, const float* k_scale,
                                           const float* v_scale, void* k_cache, void* v_cache, void* workspace,
                                           size_t workspace_bytes, dspark_stream_t stream) {
    using namespace dspark;
    if (rows < 0 || rows > 0x7fffffffll || Hkv < 1 || Hkv > 1024 || D < 8 || D > 256 || D % 8 != 0 || page < 1 ||
        num_blocks < 1)
        return DSPARK_ERR_INVALID_ARGUMENT;
    const bool scaled = cache_dt == DSPARK_E4M3 || cache_dt == DSPARK_E2M1;
    if ((dt != DSPARK_BF16 && dt != DSPARK_F32) || (cache_dt != dt && !scaled)) return DSPARK_ERR_INVALID_ARGUMENT;
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
    if (workspace_bytes < dspark_write_kv_workspace_size()) return DSPARK_ERR_WORKSPACE_TOO_SMALL;
    clear_stale_error();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) return clear_status(workspace, s);
    if (cache_dt == DSPARK_E2M1) {
        RotateArgs r{};
        r.rows = rows, r.k_stride = k_stride, r.v_stride = v_stride;
        r.slots = static_cast<int64_t>(num_blocks) * page;
        r.Hkv = Hkv, r.D = D, r.page = page, r.k = k, r.v = v, r.slot = slot, r.k_scale = k_scale, r.v_scale = v_scale;
        r.kc = k_cache, r.vc = v_cache, r.status = static_cast<StatusBlock*>(workspace);
        return launch_rotate(r, dt, cache_dt, s);
    }
    WriteArgs p{};
    p.rows = rows, p.k_stride = k_stride, p.v_stride = v_stride;
    p.slots = static_cast<int64_t>(num_blocks) * page;
    p.heads = Hkv, p.D = D, p.page = page;
    p.parts = static_cast<int>(width / 8);
    // Four rows a thread, and fewer where the rows would not fill the GPU.
    p.lanes = 1;
    while (p.lanes < kThreads && p.lanes < 2 * p.parts) p.lanes *= 2;
    const int groups = kThreads / p.lanes;
    p.rows_per_block = groups * kItems < kMaxRows ? groups * kItems : kMaxRows;
    while (p.rows_per_block > 1 && (rows + p.rows_per_block - 1) / p.rows_per_block < 2 * sm_count(current_device()))
        p.rows_per_block /= 2;
    p.alone = rows <= kAlone;
    p.k = k, p.v = v, p.slot = slot, p.k_scale = k_scale, p.v_scale = v_scale, p.kc = k_cache, p.vc = v_cache;
    p.status = static_cast<StatusBlock*>(workspace);
    const unsigned grid = static_cast<unsigned>((rows + p.rows_per_block - 1) / p.rows_per_block);
    const bool bf16 = dt == DSPARK_BF16, fp8 = cache_dt == DSPARK_E4M3;
    void (*kernel)(WriteArgs) = bf16 ? (fp8 ? write_kv<__nv_bfloat16, true> : write_kv<__nv_bfloat16, false>)
                                     : (fp8 ? write_kv<float, true> : write_kv<float, false>);
    if (p.alone) {
        kernel<<<grid, kThreads, 0, s>>>(p);
        return launch_status();
    }
    return launch_cleared(workspace, kStatusBytes, kernel, dim3(grid), kThreads, 0, s, p);
}
