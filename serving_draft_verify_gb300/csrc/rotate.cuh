// Arguments of the rotating and storing kernel (rotate.cu), for the calls that share it.
#pragma once

#include "host_common.h"
#include "kv_store.cuh"

namespace dspark {

struct RotateArgs {
    int64_t rows, q_stride, k_stride, v_stride, out_stride, slots;     // strides in elements
    int Hq, Hkv, D, rot, page;
    bool interleaved, transposed;
    const void *q, *k, *v;
    const int32_t* position;                    // NULL: no rotation
    const float* freq;
    float magnitude;
    const int64_t* slot;
    const float *k_scale, *v_scale;
    void *out, *kc, *vc;
    StatusBlock* status;
    // filled in by the launch
    int rows_per_block, units, turned;          // units of a head, and how many of them are rotated
    bool alone;                                 // no clearing came before
    Page4 g;
};

// Launches the kernel for rows of `dt` and caches of `cache_dt` (any value where Hkv is 0).
dspark_status_t launch_rotate(RotateArgs p, dspark_dtype_t dt, dspark_dtype_t cache_dt, cudaStream_t s);

}  // namespace dspark
