// dspark_adjust_logits: penalties for repeated tokens, biases and grammar masks on
// the target rows of a round.
//
// Mathematics, for token v of row k (0-based) of request b, with n(v) the times v
// stands in the request's output so far (its output tokens, then the draft's first k
// tokens) and s(v) whether it stands in the prompt or in that output:
//   y = x;  if s(v): y = y > 0 ? y / rho : y rho;
//   y -= f n(v);  if n(v) > 0: y -= p;  y += bias(v);  masked: y = -inf,
// in float32, rounded once.  A token with neither count, bias nor mask is copied
// bit for bit.
//
// Bound by memory: the rows in and out.  A block owns a piece of the vocabulary of
// one request: it counts that piece's tokens of the history in shared memory once
// and then streams the piece of every wanted row, adding one draft token between
// rows.  One 32-bit word per token holds the count, the prompt bit and the index of
// the token's bias; a bit for each token says whether its word is not zero, so that a row's
// pass is a copy with the mask's bits, and a thread goes through its set bits alone (one in a
// hundred in a long text, but nearly every warp has some: taking all eight tokens of 16
// bytes wherever one was set made the kernel issue four times as many instructions, and
// going over the copy again for a list of them cost more in scattered accesses, 396 us
// for 256 requests of up to 17 rows where this takes 314).
// Vocabularies number frequent tokens first, so the pieces with the most set bits are the
// first: blocks of one piece are neighbours in the launch, the first pieces start first, and
// the light ones fill the end.
#include "launch.cuh"

namespace dspark {
namespace {

constexpr uint32_t kCountBits = 20, kCountMask = (1u << kCountBits) - 1;
constexpr uint32_t kPrompt = 1u << kCountBits;
constexpr int kBiasShift = 21;
constexpr int kMaxBias = (1 << (32 - kBiasShift)) - 1;      // 2047
constexpr int kMaxHistory = static_cast<int>(kCountMask) - DSPARK_MAX_GAMMA;
constexpr int kThreads = 256;
constexpr int kPieceBytes = 16384;          // of a row, at most (256 requests, bf16: 314 us; with half of it 338)

struct AdjustArgs {
    int R, V, chunk, n_bias, n_mask;
    int64_t ld_history, ld_mask;
    const void* logits;
    const int32_t *ell, *history, *prompt_len, *history_len, *draft;
    const float *repetition, *frequency, *presence;
    const int32_t* bias_token;
    const float* bias_value;
    const int32_t* mask_row;
    const uint32_t* mask;
    void* out;
    StatusBlock* status;
};

// One step of the definition for a token that its word touches.
struct Rules {
    float rho, f, p;
    const float* bias;
    __device__ __forceinline__ float operator()(float x, uint32_t w) const {
        const uint32_t n = w & kCountMask;
        if ((w & (kPrompt | kCountMask)) != 0) {
            if (x > 0.f) x = __fdiv_rn(x, rho);
            else x *= rho;
        }
        if (n != 0) {
            x = __fsub_rn(x, __fmul_rn(f, static_cast<float>(n)));
            x -= p;
        }
        if ((w >> kBiasShift) != 0) x += bias[(w >> kBiasShift) - 1];
        return x;
    }
};

template <typename T>
struct Row;
template <>
struct Row<__nv_bfloat16> {
    static constexpr int kVec = 8;
    __device__ static float get(const uint4& u, int i) {
        const uint32_t w = i < 4 ? (i < 2 ? u.x : u.y) : (i < 6 ? u.z : u.w);
        return __uint_as_float((i & 1) ? w & 0xffff0000u : w << 16);
    }
    __device__ static void put(uint4& u, int i, float x) {
        const uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rn(x));
        const uint32_t keep = (i & 1) ? 0x0000ffffu : 0xffff0000u, bits = (i & 1) ? h << 16 : h;
        if ((i >> 1) == 0) u.x = (u.x & keep) | bits;
        if ((i >> 1) == 1) u.y = (u.y & keep) | bits;
        if ((i >> 1) == 2) u.z = (u.z & keep) | bits;
        if ((i >> 1) == 3) u.w = (u.w & keep) | bits;
    }
    // -inf in the place of each element whose bit of `keep` is 0
    __device__ static uint32_t masked(uint32_t w, uint32_t keep) {
        const uint32_t m = ((keep & 1u) ? 0xffffu : 0u) | ((keep & 2u) ? 0xffff0000u : 0u);
        return (w & m) | (0xFF80FF80u & ~m);
    }
    __device__ static void mask(uint4& u, uint32_t keep) {
        u.x = masked(u.x, keep);
        u.y = masked(u.y, keep >> 2);
        u.z = masked(u.z, keep >> 4);
        u.w = masked(u.w, keep >> 6);
    }
};
template <>
struct Row<float> {
    static constexpr int kVec = 4;
    __device__ static float get(const uint4& u, int i) {
        return __uint_as_float(i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w);
    }
    __device__ static void put(uint4& u, int i, float x) {
        if (i == 0) u.x = __float_as_uint(x);
        if (i == 1) u.y = __float_as_uint(x);
        if (i == 2) u.z = __float_as_uint(x);
        if (i == 3) u.w = __float_as_uint(x);
    }
    __device__ static void mask(uint4& u, uint32_t keep) {
        u.x = (keep & 1u) ? u.x : 0xFF800000u;
        u.y = (keep & 2u) ? u.y : 0xFF800000u;
        u.z = (keep & 4u) ? u.z : 0xFF800000u;
        u.w = (keep & 8u) ? u.w : 0xFF800000u;
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) adjust_logits(AdjustArgs p) {
    constexpr int kVec = Row<T>::kVec, kUnroll = 2;
    extern __shared__ uint32_t words[];                     // [chunk], the biases [n_bias], the bits [chunk / kVec bytes]
    float* s_bias = reinterpret_cast<float*>(words + p.chunk);
    uint8_t* flags = reinterpret_cast<uint8_t*>(s_bias + p.n_bias);
    __shared__ int s_draft[DSPARK_MAX_GAMMA];
    const int b = blockIdx.x, tid = threadIdx.x;
    const int v0 = blockIdx.y * p.chunk;
    const int nv = min(p.chunk, p.V - v0);
    // Every block of a request sees the same errors; the first piece's tells them.  Where there is one
    // request that block clears the status as well, and nothing has to come before.
    StatusBlock* status = blockIdx.y == 0 ? p.status : nullptr;
    if (gridDim.x == 1 && blockIdx.y == 0) {
        if (tid < 4) reinterpret_cast<uint32_t*>(status)[tid] = 0;
        __syncthreads();
    }
    int rows = p.R;
    if (p.ell != nullptr) {
        const int e = p.ell[b];
        if (e < 0 || e >= p.R) {
            if (tid == 0) tell(status, DSPARK_ERR_DEVICE_CHECK, 1);        // waits for the clearing too
            return;
        }
        rows = e + 1;
    }
    // The stream: batches of kUnroll pieces a thread, row by row.  A batch is loaded while the one
    // before is worked on, and the first while the history is counted.
    const int nvec = nv / kVec;
    struct Batch {
        uint4 x[kUnroll];
        uint32_t keep[kUnroll];
        bool masked;
    };
    auto mask_of = [&](int k) {
        int mr = p.mask_row != nullptr ? __ldg(p.mask_row + static_cast<int64_t>(b) * p.R + k) : -1;
        return mr < -1 || mr >= p.n_mask ? -1 : mr;
    };
    int next_mask = mask_of(0);                             // of the row being loaded
    auto load = [&](Batch& t, int k, int i0) {
        const uint4* in = reinterpret_cast<const uint4*>(static_cast<const T*>(p.logits) + (static_cast<int64_t>(b) * p.R + k) * p.V + v0);
        const uint32_t* mask = p.mask + next_mask * p.ld_mask + v0 / 32;
        t.masked = next_mask >= 0;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * kThreads;
            t.keep[u] = 0xffffffffu;
            if (i < nvec) {
                t.x[u] = __ldcs(in + i);
                if (t.masked) t.keep[u] = __ldg(mask + i * kVec / 32) >> (i * kVec % 32);
            }
        }
    };
    Batch one, two;                                         // by turns
    load(one, 0, tid);
    for (int i = tid; i < p.chunk / 4; i += kThreads) reinterpret_cast<uint4*>(words)[i] = make_uint4(0, 0, 0, 0);
    if (tid < rows) {
        // the draft token that the row's count gains
        int t = -1;
        if (tid > 0 && p.draft != nullptr) {
            t = p.draft[static_cast<int64_t>(b) * (p.R - 1) + tid - 1];
            if (t < 0 || t >= p.V) tell(status, DSPARK_ERR_DEVICE_CHECK, 3);
            t = t >= v0 && t < v0 + nv ? t - v0 : -1;
        }
        if (tid > 0) s_draft[tid - 1] = t;
        if (p.mask_row != nullptr) {
            const int mr = p.mask_row[static_cast<int64_t>(b) * p.R + tid];
            if (mr < -1 || mr >= p.n_mask) tell(status, DSPARK_ERR_DEVICE_CHECK, 5);
        }
    }
    __syncthreads();

    // the history's tokens of this piece
    const int32_t* hist = p.history + static_cast<int64_t>(b) * p.ld_history;
    int hn = p.history_len != nullptr ? p.history_len[b] : 0, pn = p.prompt_len != nullptr ? p.prompt_len[b] : 0;
    if (hn < 0 || hn > p.ld_history || pn < 0 || pn > hn) {
        if (tid == 0) tell(status, DSPARK_ERR_DEVICE_CHECK, 2);
        hn = pn = 0;
    }
    auto count = [&](int i, int t) {
        const int v = t - v0;
        if (t < 0 || t >= p.V) tell(status, DSPARK_ERR_DEVICE_CHECK, 3);
        else if (v >= 0 && v < nv) {
            if (i < pn) atomicOr(&words[v], kPrompt);
            else atomicAdd(&words[v], 1u);
        }
    };
    // sixteen tokens a thread at a time where the rows allow 16-byte loads: every piece reads the whole
    // history, and what that costs a block is its latency
    int done = 0;
    if ((reinterpret_cast<uintptr_t>(hist) & 15) == 0) {
        done = hn & ~3;
        for (int i0 = 4 * tid; i0 < done; i0 += 16 * kThreads) {
            int4 t[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + 4 * j * kThreads < done) t[j] = __ldg(reinterpret_cast<const int4*>(hist + i0 + 4 * j * kThreads));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + 4 * j * kThreads;
                if (i >= done) continue;
                count(i, t[j].x);
                count(i + 1, t[j].y);
                count(i + 2, t[j].z);
                count(i + 3, t[j].w);
            }
        }
    }
    for (int i = done + tid; i < hn; i += kThreads) count(i, hist[i]);
    // the biases: the first entry of a token sums those of all its entries, in order
    for (int i = tid; i < p.n_bias; i += kThreads) {
        const int32_t* tok = p.bias_token + static_cast<int64_t>(b) * p.n_bias;
        const float* val = p.bias_value + static_cast<int64_t>(b) * p.n_bias;
        const int t = tok[i], v = t - v0;
        if (t < -1 || t >= p.V) tell(status, DSPARK_ERR_DEVICE_CHECK, 4);
        if (t < 0 || v < 0 || v >= nv) continue;
        bool first = true;
        for (int j = 0; j < i && first; ++j) first = tok[j] != t;
        if (!first) continue;
        float sum = val[i];
        for (int j = i + 1; j < p.n_bias; ++j)
            if (tok[j] == t) sum += val[j];
        s_bias[i] = sum;
        atomicOr(&words[v], static_cast<uint32_t>(i + 1) << kBiasShift);
    }
    const Rules rules{p.repetition != nullptr ? p.repetition[b] : 1.f, p.frequency != nullptr ? p.frequency[b] : 0.f,
                      p.presence != nullptr ? p.presence[b] : 0.f, s_bias};
    __syncthreads();
    for (int i = tid; i < p.chunk / kVec; i += kThreads) {
        uint32_t any = 0;
#pragma unroll
        for (int j = 0; j < kVec; j += 4) {
            const uint4 w = reinterpret_cast<const uint4*>(words)[(i * kVec + j) / 4];
            any |= ((w.x != 0) | (w.y != 0) << 1 | (w.z != 0) << 2 | (w.w != 0) << 3) << j;
        }
        flags[i] = static_cast<uint8_t>(any);
    }
    __syncthreads();

    // A batch's work, once the next one's loads are on their way; false after the last.
    int k = 0, i0 = tid;
    auto work = [&](Batch& now, Batch& then) -> bool {
        const int at = i0, row = k;
        i0 += kUnroll * kThreads;
        if (i0 - tid >= nvec) {
            i0 = tid;
            ++k;
            if (k < rows) next_mask = mask_of(k);
        }
        if (k < rows) load(then, k, i0);
        if (at == tid && row > 0) {
            const int t = s_draft[row - 1];
            if (t >= 0) {
                __syncthreads();                            // the row before has been done with the old count
                if (tid == 0) {
                    words[t] += 1;
                    flags[t / kVec] |= static_cast<uint8_t>(1u << (t % kVec));
                }
                __syncthreads();
            }
        }
        uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (static_cast<int64_t>(b) * p.R + row) * p.V + v0);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = at + u * kThreads;
            if (i >= nvec) continue;
            // what the mask hides needs no rules
            for (uint32_t set = flags[i] & now.keep[u]; set != 0; set &= set - 1) {
                const int j = __ffs(set) - 1;
                Row<T>::put(now.x[u], j, rules(Row<T>::get(now.x[u], j), words[i * kVec + j]));
            }
            if (now.masked) Row<T>::mask(now.x[u], now.keep[u]);
            __stcs(out + i, now.x[u]);
        }
        return k < rows;
    };
    while (work(one, two) && work(two, one)) {
    }
    if (blockIdx.x == 0) head_cleared();
}

}  // namespace
}  // namespace dspark

extern "C" size_t dspark_adjust_logits_workspace_size(void) { return dspark::kStatusBytes; }

extern "C" dspark_status_t dspark_adjust_logits(int B, int R, int V, dspark_dtype_t dt, const void* logits,
                                                const int32_t* ell, const int32_t* history, int64_t ld_history,
                                                const int32_t* prompt_len, const int32_t* history_len,
                                                const int32_t* draft, const float* repetition, const float* frequency,
                                                const float* presence, const int32_t* bias_token,
                                                const float* bias_value, int n_bias, const int32_t* mask_row,
                                                const uint32_t* mask, int n_mask, int64_t ld_mask, void* out,
                                                void* workspace, size_t workspace_bytes, dspark_stream_t stream) {
    using namespace dspark;
    if (B < 1 || B > 65535 || R < 1 || R > DSPARK_MAX_GAMMA + 1 || V < 1) return DSPARK_ERR_INVALID_ARGUMENT;
    if ((dt != DSPARK_BF16 && dt != DSPARK_F32) || V % (dt == DSPARK_BF16 ? 8 : 4) != 0)
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (logits == nullptr || out == nullptr || !aligned16(logits) || !aligned16(out)) return DSPARK_ERR_INVALID_ARGUMENT;
    // a history of no columns has no address; its lengths are checked on the device like any others
    const bool has_history = history != nullptr || (history_len != nullptr && ld_history == 0);
    if (has_history != (history_len != nullptr) || (prompt_len != nullptr && !has_history) || ld_history < 0)
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (n_bias < 0 || (n_bias > 0 && (bias_token == nullptr || bias_value == nullptr)))
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (mask_row != nullptr && (n_mask < 0 || (n_mask > 0 && mask == nullptr) || ld_mask < (V + 31) / 32))
        return DSPARK_ERR_INVALID_ARGUMENT;
    if (n_bias > kMaxBias || ld_history > kMaxHistory) return DSPARK_ERR_UNSUPPORTED;
    if (workspace == nullptr || !aligned256(workspace)) return DSPARK_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < dspark_adjust_logits_workspace_size()) return DSPARK_ERR_WORKSPACE_TOO_SMALL;
    // in place or apart: partly overlapping rows would be read after they were written
    const size_t bytes = static_cast<size_t>(B) * R * V * (dt == DSPARK_BF16 ? 2 : 4);
    const uintptr_t a = reinterpret_cast<uintptr_t>(logits), o = reinterpret_cast<uintptr_t>(out);
    if (a != o && a < o + bytes && o < a + bytes) return DSPARK_ERR_INVALID_ARGUMENT;
    clear_stale_error();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    AdjustArgs p{R,        V,     kPieceBytes / (dt == DSPARK_BF16 ? 2 : 4), n_bias,      n_mask,      ld_history, ld_mask,
                 logits,   ell,   history,       prompt_len,  history_len, draft,      repetition,
                 frequency, presence, bias_token, bias_value, mask_row,    mask,       out,
                 static_cast<StatusBlock*>(workspace)};
    while (p.chunk > 1024 && static_cast<int64_t>(B) * ((V + p.chunk - 1) / p.chunk) < 4 * sm_count(current_device()))
        p.chunk /= 2;
    const dim3 grid(B, (V + p.chunk - 1) / p.chunk);
    const size_t smem = p.chunk * 4 + static_cast<size_t>(n_bias) * 4 + p.chunk / 4;
    if (B == 1) {
        if (dt == DSPARK_BF16) adjust_logits<__nv_bfloat16><<<grid, kThreads, smem, s>>>(p);
        else adjust_logits<float><<<grid, kThreads, smem, s>>>(p);
        return launch_status();
    }
    return launch_cleared(workspace, kStatusBytes, dt == DSPARK_BF16 ? adjust_logits<__nv_bfloat16> : adjust_logits<float>,
                          grid, kThreads, smem, s, p);
}
