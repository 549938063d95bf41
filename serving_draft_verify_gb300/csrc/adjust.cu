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
// the token's bias; a word of zero means the token passes unchanged.
#include "common.cuh"
#include "host_common.h"

namespace dspark {
namespace {

constexpr uint32_t kCountBits = 20, kCountMask = (1u << kCountBits) - 1;
constexpr uint32_t kPrompt = 1u << kCountBits;
constexpr int kBiasShift = 21;
constexpr int kMaxBias = (1 << (32 - kBiasShift)) - 1;      // 2047
constexpr int kMaxHistory = static_cast<int>(kCountMask) - DSPARK_MAX_GAMMA;
constexpr int kThreads = 256;

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

// One step of the definition for a token that its word or its mask bit touches.
struct Rules {
    float rho, f, p;
    const float* bias;
    __device__ __forceinline__ float operator()(float x, uint32_t w, bool keep) const {
        if (!keep) return -__uint_as_float(0x7f800000u);
        const uint32_t n = w & kCountMask;
        if ((w & (kPrompt | kCountMask)) != 0) x = x > 0.f ? __fdiv_rn(x, rho) : x * rho;
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
        const uint32_t w = i < 2 ? u.x : i < 4 ? u.y : i < 6 ? u.z : u.w;
        return (i & 1) ? bf16hi(w) : bf16lo(w);
    }
    __device__ static void put(uint4& u, int i, float x) {
        const uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rn(x));
        uint32_t& w = i < 2 ? u.x : i < 4 ? u.y : i < 6 ? u.z : u.w;
        w = (i & 1) ? (w & 0xffffu) | (h << 16) : (w & 0xffff0000u) | h;
    }
};
template <>
struct Row<float> {
    static constexpr int kVec = 4;
    __device__ static float get(const uint4& u, int i) {
        return __uint_as_float(i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w);
    }
    __device__ static void put(uint4& u, int i, float x) {
        uint32_t& w = i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
        w = __float_as_uint(x);
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) adjust_logits(AdjustArgs p) {
    extern __shared__ uint32_t words[];                     // [chunk], then the biases [n_bias]
    float* s_bias = reinterpret_cast<float*>(words + p.chunk);
    constexpr int kVec = Row<T>::kVec;
    const int b = blockIdx.y, tid = threadIdx.x;
    const int v0 = blockIdx.x * p.chunk;
    const int nv = min(p.chunk, p.V - v0);
    int rows = p.R;
    if (p.ell != nullptr) {
        const int e = p.ell[b];
        if (e < 0 || e >= p.R) {
            if (tid == 0) set_status(p.status, DSPARK_ERR_DEVICE_CHECK, 1);
            return;
        }
        rows = e + 1;
    }
    for (int i = tid; i < p.chunk; i += kThreads) words[i] = 0;
    __syncthreads();

    // the history's tokens of this piece
    const int32_t* hist = p.history + static_cast<int64_t>(b) * p.ld_history;
    int hn = p.history_len != nullptr ? p.history_len[b] : 0, pn = p.prompt_len != nullptr ? p.prompt_len[b] : 0;
    if (hn < 0 || hn > p.ld_history || pn < 0 || pn > hn) {
        if (tid == 0) set_status(p.status, DSPARK_ERR_DEVICE_CHECK, 2);
        hn = pn = 0;
    }
    for (int i = tid; i < hn; i += kThreads) {
        const int t = hist[i];
        if (t < 0 || t >= p.V) {
            set_status(p.status, DSPARK_ERR_DEVICE_CHECK, 3);
            continue;
        }
        const int v = t - v0;
        if (v < 0 || v >= nv) continue;
        if (i < pn) atomicOr(&words[v], kPrompt);
        else atomicAdd(&words[v], 1u);
    }
    // the biases: the first entry of a token sums those of all its entries, in order
    for (int i = tid; i < p.n_bias; i += kThreads) {
        const int32_t* tok = p.bias_token + static_cast<int64_t>(b) * p.n_bias;
        const float* val = p.bias_value + static_cast<int64_t>(b) * p.n_bias;
        const int t = tok[i], v = t - v0;
        if (t < -1 || t >= p.V) set_status(p.status, DSPARK_ERR_DEVICE_CHECK, 4);
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
    Rules rules{p.repetition != nullptr ? p.repetition[b] : 1.f, p.frequency != nullptr ? p.frequency[b] : 0.f,
                p.presence != nullptr ? p.presence[b] : 0.f, s_bias};

    for (int k = 0; k < rows; ++k) {
        __syncthreads();
        if (k > 0 && p.draft != nullptr) {
            if (tid == 0) {
                const int t = p.draft[static_cast<int64_t>(b) * (p.R - 1) + k - 1];
                if (t < 0 || t >= p.V) set_status(p.status, DSPARK_ERR_DEVICE_CHECK, 3);
                else if (t >= v0 && t < v0 + nv) words[t - v0] += 1;
            }
            __syncthreads();
        }
        const int64_t row = static_cast<int64_t>(b) * p.R + k;
        int mr = p.mask_row != nullptr ? p.mask_row[row] : -1;
        if (mr < -1 || mr >= p.n_mask) {
            if (tid == 0) set_status(p.status, DSPARK_ERR_DEVICE_CHECK, 5);
            mr = -1;
        }
        const uint32_t* mask = mr >= 0 ? p.mask + mr * p.ld_mask : nullptr;
        const uint4* in = reinterpret_cast<const uint4*>(static_cast<const T*>(p.logits) + row * p.V + v0);
        uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + row * p.V + v0);
        for (int i = tid; i < nv / kVec; i += kThreads) {
            uint4 x = in[i];
            uint32_t keep = 0xffffffffu;
            if (mask != nullptr) keep = mask[(v0 + i * kVec) >> 5] >> ((v0 + i * kVec) & 31);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const uint32_t w = words[i * kVec + j];
                const bool ok = ((keep >> j) & 1u) != 0;
                if (w != 0 || !ok) Row<T>::put(x, j, rules(Row<T>::get(x, j), w, ok));
            }
            out[i] = x;
        }
    }
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
    if ((history == nullptr) != (history_len == nullptr) || (prompt_len != nullptr && history == nullptr) ||
        ld_history < 0)
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
    if (clear_status(workspace, s) != DSPARK_OK) return DSPARK_ERR_CUDA;
    AdjustArgs p{R,        V,     4096,          n_bias,      n_mask,      ld_history, ld_mask,
                 logits,   ell,   history,       prompt_len,  history_len, draft,      repetition,
                 frequency, presence, bias_token, bias_value, mask_row,    mask,       out,
                 static_cast<StatusBlock*>(workspace)};
    while (p.chunk > 1024 && static_cast<int64_t>(B) * ((V + p.chunk - 1) / p.chunk) < 4 * sm_count(current_device()))
        p.chunk /= 2;
    const dim3 grid((V + p.chunk - 1) / p.chunk, B);
    const size_t smem = p.chunk * 4 + static_cast<size_t>(n_bias) * 4;
    if (dt == DSPARK_BF16) adjust_logits<__nv_bfloat16><<<grid, kThreads, smem, s>>>(p);
    else adjust_logits<float><<<grid, kThreads, smem, s>>>(p);
    return launch_status();
}
