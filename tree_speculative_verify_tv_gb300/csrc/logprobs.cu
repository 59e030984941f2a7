// logprobs.cu -- log probabilities of given tokens, entropy and the most likely tokens.
//
//   m = max s x, z = sum e^{s x - m};  logprob = s x_t - m - ln z;
//   entropy = ln z - (sum e^{s x - m} (s x - m)) / z
#include "tv_internal.cuh"

namespace tv {
namespace {

constexpr int kThreadsLp = 256;

// Order of logits: larger value, larger key; a NaN above all, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

template <typename E>
__global__ void __launch_bounds__(kThreadsLp) logprobs_kernel(LogprobsArgs a) {
    __shared__ float s_f[2][kThreadsLp / 32];
    __shared__ unsigned long long s_k[kThreadsLp / 32 + 1];
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    pdl_wait();
    pdl_launch_next();
    int row = a.rows ? a.rows[r] : r;
    int token = a.tokens ? a.tokens[r] : -1;
    if (tid == 0 && (row >= a.N || token >= a.V)) report(a.status, TV_ERR_SHAPE);
    if (row < 0 || row >= a.N) {
        if (tid == 0) {
            if (a.logprob) a.logprob[r] = 0.f;
            if (a.entropy) a.entropy[r] = 0.f;
        }
        for (int i = tid; i < a.top; i += kThreadsLp) {
            a.top_token[(size_t)r * a.top + i] = -1;
            a.top_logprob[(size_t)r * a.top + i] = 0.f;
        }
        return;
    }
    const E *x = static_cast<const E *>(a.logits) + (size_t)row * a.stride;
    float m = -INFINITY;
    bool bad = false;
    for (int i = tid; i < a.V; i += kThreadsLp) {
        const float y = to_f32(x[i]) * a.scale;
        bad |= !(y < INFINITY);
        m = fmaxf(m, y);
    }
    bad = __syncthreads_or(bad);
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) s_f[0][warp] = m;
    __syncthreads();
    for (int i = 0; i < kThreadsLp / 32; ++i) m = fmaxf(m, s_f[0][i]);
    __syncthreads();
    float z = 0.f, t = 0.f;
    if (m > -INFINITY)
        for (int i = tid; i < a.V; i += kThreadsLp) {
            const float y = to_f32(x[i]) * a.scale - m, e = expf(y);
            z += e;
            if (e > 0.f) t += e * y;
        }
    z = warp_sum(z);
    t = warp_sum(t);
    if (lane == 0) {
        s_f[0][warp] = z;
        s_f[1][warp] = t;
    }
    __syncthreads();
    z = t = 0.f;
    for (int i = 0; i < kThreadsLp / 32; ++i) {
        z += s_f[0][i];
        t += s_f[1][i];
    }
    const float lnz = logf(z);
    const auto logprob = [&](float v) {
        if (bad) return __int_as_float(0x7fffffff);
        return m > -INFINITY ? v * a.scale - m - lnz : -INFINITY;
    };
    if (tid == 0) {
        if (a.logprob)
            a.logprob[r] = token >= 0 && token < a.V ? logprob(to_f32(x[token])) : 0.f;
        if (a.entropy)
            a.entropy[r] = bad ? __int_as_float(0x7fffffff) : m > -INFINITY ? lnz - t / z : 0.f;
    }
    unsigned long long last = ~0ull;
    for (int j = 0; j < a.top; ++j) {
        unsigned long long best = 0;
        for (int i = tid; i < a.V; i += kThreadsLp) {
            const unsigned long long k =
                ((unsigned long long)order_key(to_f32(x[i])) << 32) | (0xffffffffu - i);
            if (k < last && k > best) best = k;
        }
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long k = __shfl_xor_sync(0xffffffffu, best, o);
            best = k > best ? k : best;
        }
        if (lane == 0) s_k[warp] = best;
        __syncthreads();
        if (tid == 0) {
            for (int i = 0; i < kThreadsLp / 32; ++i) best = s_k[i] > best ? s_k[i] : best;
            const int i = (int)(0xffffffffu - (uint32_t)best);
            a.top_token[(size_t)r * a.top + j] = i;
            a.top_logprob[(size_t)r * a.top + j] = logprob(to_f32(x[i]));
            s_k[kThreadsLp / 32] = best;
        }
        __syncthreads();
        last = s_k[kThreadsLp / 32];
    }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsArgs &a, cudaStream_t s) {
    if (a.dtype == TV_BF16)
        return launch_pdl(logprobs_kernel<__nv_bfloat16>, dim3((unsigned)a.R), dim3(kThreadsLp), 0,
                          s, a);
    return launch_pdl(logprobs_kernel<float>, dim3((unsigned)a.R), dim3(kThreadsLp), 0, s, a);
}

}  // namespace tv
