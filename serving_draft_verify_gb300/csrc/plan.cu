// dspark_plan_rows: pages, positions and cache slots of the rows a step adds.
//
// Mathematics, with page size P, base_b = len_b + advance_b, need_b =
// ceil((base_b + rows_b) / P), take_b = max(0, need_b - held_b) and give_b =
// max(0, held_b - need_b): exclusive prefix sums of rows, take and give over
// the requests name every row's place in the step, the ring entry of every
// new page and the ring place of every page that goes back.
//
// One launch.  Every block runs the prefix sums over all B requests itself (they
// are a few kilobytes that L2 holds), so no block waits for another, and keeps
// the part that its own rows need (a thread a row): the first row of each request marks
// its place in shared memory and a running maximum over the marks gives every row its
// request.  A new page starts at a row of the step, so the thread of that row
// enters it in the table; pages that go back are copied by the block that owns the
// request's tile.  The last block to finish (a counter, nobody waits) writes the
// per-request state, so the state may be updated in place.
//
// Bound by latency (16 bytes a row and a few words a request move): a call in a graph takes 3.5 us
// for 16 requests (one block of 256 threads) and 9.8 us for 1024 requests with 20,000 rows.
#include "launch.cuh"

namespace dspark {
namespace {

struct PlanArgs {
    int B, page, max_blocks, num_blocks;
    int64_t room, ld;
    const int32_t *len, *advance, *rows, *held, *free_state;
    int32_t* ring;
    int32_t* table;
    int32_t *len_out, *held_out, *free_out, *row_offset, *row_request, *position;
    int64_t* slot;
    StatusBlock* status;
    uint32_t* ticket;
};

// What one request asks for; `bad` is 1 or 2, the detail code of an inconsistent one.
struct Ask {
    int base, rows, held, need;
    uint32_t bad;
};

__device__ __forceinline__ Ask ask_of(const PlanArgs& p, int b) {
    Ask a{};
    const int64_t len = p.len[b];
    const int64_t adv = p.advance != nullptr ? p.advance[b] : 0;
    const int64_t rows = p.rows[b], held = p.held[b];
    const int64_t base = len + adv, end = base + rows;
    const int64_t room = static_cast<int64_t>(p.max_blocks) * p.page;
    if (len < 0 || adv < 0 || rows < 0 || held < 0 || held > p.max_blocks || base > held * p.page) {
        a.bad = 1;
        return a;
    }
    if (end > room) {
        a.bad = 2;
        return a;
    }
    a.base = static_cast<int>(base);
    a.rows = static_cast<int>(rows);
    a.held = static_cast<int>(held);
    a.need = static_cast<int>((static_cast<uint32_t>(end) + p.page - 1) / static_cast<uint32_t>(p.page));
    return a;
}

// Exclusive prefix over the block of two 64-bit sums; the totals come back too.
struct Sums {
    unsigned long long rows, pages;      // pages: take in the low half, give in the high half
};
__device__ __forceinline__ Sums warp_scan(Sums v) {          // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long r = __shfl_up_sync(0xffffffffu, v.rows, o);
        const unsigned long long g = __shfl_up_sync(0xffffffffu, v.pages, o);
        if (lane >= o) {
            v.rows += r;
            v.pages += g;
        }
    }
    return v;
}
// warp_tot: kT / 32 + 1 entries, the last for the total
template <int kT>
__device__ __forceinline__ Sums block_scan(Sums v, Sums* warp_tot, Sums& total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const Sums inc = warp_scan(v);
    __syncthreads();                      // the last scan's totals have been read
    if (lane == 31) warp_tot[w] = inc;
    __syncthreads();
    if (w == 0) {
        const Sums t = lane < kT / 32 ? warp_tot[lane] : Sums{0, 0};
        const Sums all = warp_scan(t);
        if (lane < kT / 32) warp_tot[lane] = Sums{all.rows - t.rows, all.pages - t.pages};
        if (lane == 31) warp_tot[kT / 32] = all;
    }
    __syncthreads();
    const Sums before = warp_tot[w];
    total = warp_tot[kT / 32];
    return Sums{before.rows + inc.rows - v.rows, before.pages + inc.pages - v.pages};
}
// x modulo cap for 0 <= x < 3 cap.
__device__ __forceinline__ int64_t around(int64_t x, int cap) {
    x = x >= cap ? x - cap : x;
    return x >= cap ? x - cap : x;
}

template <int kT>
__global__ void __launch_bounds__(kT) plan_rows(PlanArgs p) {
    __shared__ Sums warp_tot[kT / 32 + 1];
    __shared__ int s_mark[kT];            // marked row -> request + 1
    __shared__ int s_pos[kT], s_held[kT];
    __shared__ long long s_take[kT];
    __shared__ int s_gb[kT], s_gneed[kT], s_gheld[kT];
    __shared__ long long s_gat[kT];
    __shared__ int s_ngive, s_last;
    __shared__ int warp_max_mark[kT / 32];

    const int tid = threadIdx.x;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kT;
    s_mark[tid] = 0;
    if (tid == 0) s_ngive = 0;
    if (gridDim.x == 1 && tid < 4) reinterpret_cast<uint32_t*>(p.status)[tid] = 0;   // alone: no clear came before
    __syncthreads();

    const int head = p.free_state[0], count = p.free_state[1];
    const int tiles = (p.B + kT - 1) / kT;
    Sums run{0, 0};
    uint32_t bad = 0;                     // bit d - 1: a request of this thread is refused with detail d
    Ask own{};                            // this thread's request of the last tile, kept for the state write
    Sums own_at{0, 0};
    for (int t = 0; t < tiles; ++t) {
        const int b = t * kT + tid;
        Ask a{};
        if (b < p.B) a = ask_of(p, b);
        bad |= a.bad;
        const int take = a.need > a.held ? a.need - a.held : 0, give = a.held > a.need ? a.held - a.need : 0;
        Sums v{static_cast<unsigned long long>(a.rows),
               static_cast<unsigned long long>(take) | (static_cast<unsigned long long>(give) << 32)};
        Sums tot;
        Sums at = block_scan<kT>(v, warp_tot, tot);
        at.rows += run.rows;
        at.pages += run.pages;
        run.rows += tot.rows;
        run.pages += tot.pages;
        own = a;
        own_at = at;
        const int64_t start = static_cast<int64_t>(at.rows);
        if (a.rows > 0 && start < r0 + kT && start + a.rows > r0) {
            const int m = start > r0 ? static_cast<int>(start - r0) : 0;
            s_mark[m] = b + 1;
            s_pos[m] = a.base + static_cast<int>(r0 + m - start);
            s_held[m] = a.held;
            s_take[m] = static_cast<long long>(at.pages & 0xffffffffu);
        }
        if (t == static_cast<int>(blockIdx.x) && give > 0) {
            const int e = atomicAdd(&s_ngive, 1);
            s_gb[e] = b;
            s_gneed[e] = a.need;
            s_gheld[e] = a.held;
            s_gat[e] = static_cast<long long>(at.pages >> 32);
        }
    }
    const int64_t N = static_cast<int64_t>(run.rows);
    const int64_t T = static_cast<int64_t>(run.pages & 0xffffffffu), R = static_cast<int64_t>(run.pages >> 32);
    // all or nothing: every block comes to the same verdict
    const int cap = p.num_blocks;
    if (head < 0 || head >= cap || count < 0 || count > cap) bad |= 1u;
    uint32_t why = 0;
    if (__syncthreads_or(bad & 1u)) why = 1;
    else if (__syncthreads_or(bad & 2u)) why = 2;
    else if (T > count) why = 3;
    else if (count + R > cap) why = 1;
    else if (N > p.room) why = 4;
    if (why != 0 && blockIdx.x == 0 && tid == 0) tell(p.status, DSPARK_ERR_DEVICE_CHECK, why);

    // the block's rows
    const int64_t row = r0 + tid;
    int m = s_mark[tid] != 0 ? tid : -1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = max(m, __shfl_up_sync(0xffffffffu, m, o));   // own value where there is none
    if ((tid & 31) == 31) warp_max_mark[tid >> 5] = m;
    __syncthreads();
    for (int w = 0; w < (tid >> 5); ++w) m = max(m, warp_max_mark[w]);
    if (row < p.room) {
        int req = -1, pos = -1;
        int64_t slot = -1;
        if (why == 0 && row < N && m >= 0) {
            req = s_mark[m] - 1;
            pos = s_pos[m] + (tid - m);
            const int block = pos / p.page, off = pos - block * p.page, held = s_held[m];
            int32_t* entry = p.table + static_cast<int64_t>(req) * p.ld + block;
            int id;
            if (block >= held) {
                id = p.ring[around(head + s_take[m] + (block - held), cap)];
                if (off == 0) *entry = id;
            } else {
                id = *entry;
            }
            if (id < 0 || id >= cap)
                tell(p.status, DSPARK_ERR_DEVICE_CHECK, 5);
            else
                slot = static_cast<int64_t>(id) * p.page + off;
        }
        p.row_request[row] = req;
        p.position[row] = pos;
        p.slot[row] = slot;
    }
    // pages that go back, a warp to a request
    if (why == 0) {
        for (int e = tid >> 5; e < s_ngive; e += kT / 32) {
            const int need = s_gneed[e], held = s_gheld[e];
            const int32_t* from = p.table + static_cast<int64_t>(s_gb[e]) * p.ld;
            const int64_t to = static_cast<int64_t>(head) + count + s_gat[e];
            for (int j = need + (tid & 31); j < held; j += 32) p.ring[around(to + (j - need), cap)] = from[j];
        }
    }

    // the last block writes the state: by then every block has read it
    if (gridDim.x > 1) {
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            head_cleared();
            s_last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
        }
        __syncthreads();
        if (!s_last) return;
        __threadfence();
    } else {
        __syncthreads();
    }
    run = Sums{0, 0};
    for (int t = 0; t < tiles; ++t) {
        const int b = t * kT + tid;
        if (tiles > 1) {
            own = Ask{};
            if (b < p.B) own = ask_of(p, b);
            Sums tot;
            own_at = block_scan<kT>(Sums{static_cast<unsigned long long>(own.rows), 0}, warp_tot, tot);
            own_at.rows += run.rows;
            run.rows += tot.rows;
        }
        if (b < p.B) {
            p.row_offset[b] = why == 0 ? static_cast<int32_t>(own_at.rows) : 0;
            p.len_out[b] = why == 0 ? own.base : p.len[b];
            p.held_out[b] = why == 0 ? own.need : p.held[b];
        }
    }
    if (tid == 0) {
        p.row_offset[p.B] = why == 0 ? static_cast<int32_t>(N) : 0;
        p.free_out[0] = why == 0 ? static_cast<int32_t>(around(head + T, cap)) : head;
        p.free_out[1] = why == 0 ? static_cast<int32_t>(count - T + R) : count;
    }
}

}  // namespace
}  // namespace dspark

extern "C" size_t dspark_plan_rows_workspace_size(int B, int64_t max_rows) {
    (void)B;
    (void)max_rows;
    return 2 * dspark::kStatusBytes;
}

extern "C" dspark_status_t dspark_plan_rows(int B, int page, int max_blocks, int num_blocks, int64_t max_rows,
                                            const int32_t* len, const int32_t* advance, const int32_t* rows,
                                            const int32_t* held, const int32_t* free_state, int32_t* free_ring,
                                            int32_t* block_table, int64_t ld_table, int32_t* len_out,
                                            int32_t* held_out, int32_t* free_state_out, int32_t* row_offset,
                                            int32_t* row_request, int32_t* position, int64_t* slot, void* workspace,
                                            size_t workspace_bytes, dspark_stream_t stream) {
    using namespace dspark;
    if (B < 1 || B > 65535 || page < 1 || max_blocks < 1 || num_blocks < 1 || max_rows < 0 ||
        max_rows > 0x7fffffffll || ld_table < max_blocks)
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (len == nullptr || rows == nullptr || held == nullptr || free_state == nullptr || free_ring == nullptr ||
        block_table == nullptr || len_out == nullptr || held_out == nullptr || free_state_out == nullptr ||
        row_offset == nullptr || (max_rows > 0 && (row_request == nullptr || position == nullptr || slot == nullptr)))
        return DSPARK_ERR_INVALID_ARGUMENT;
    // positions are 32-bit, and so are the sums of pages over the requests
    if (static_cast<int64_t>(max_blocks) * page > 0x7fffffffll || static_cast<int64_t>(max_blocks) * B > 0x7fffffffll)
        return DSPARK_ERR_UNSUPPORTED;
    if (workspace == nullptr || !aligned256(workspace)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < dspark_plan_rows_workspace_size(B, max_rows)) return DSPARK_ERR_WORKSPACE_TOO_SMALL;
    clear_stale_error();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    PlanArgs p{B,        page,      max_blocks, num_blocks,     max_rows, ld_table, len,         advance,
               rows,     held,      free_state, free_ring,      block_table, len_out, held_out,  free_state_out,
               row_offset, row_request, position, slot,         static_cast<StatusBlock*>(workspace),
               reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + kStatusBytes)};
    // a small step is one small block: its scans and barriers are the call's time (16 requests in a graph:
    // 3.5 us, with the large block 4.4)
    const bool small = B <= 256 && max_rows <= 256;
    const int64_t tile = small ? 256 : 1024;
    const int64_t row_tiles = (max_rows + tile - 1) / tile, req_tiles = (B + tile - 1) / tile;
    const int64_t grid = row_tiles > req_tiles ? row_tiles : req_tiles;
    if (grid > 1)
        return launch_cleared(workspace, kStatusBytes + 16, plan_rows<1024>, dim3(static_cast<unsigned>(grid)), 1024, 0, s, p);
    if (small) plan_rows<256><<<1, 256, 0, s>>>(p);
    else plan_rows<1024><<<1, 1024, 0, s>>>(p);
    return launch_status();
}
