// qk_norm_rope.cu -- queries and keys of an attention layer normed per head and rotated at
// their positions, in one pass.
//
//   y_c = x_c w_c / sqrt(mean x^2 + eps);  (a, b) -> (a cos t - b sin t, b cos t + a sin t)
// A tree node stands at the position that tree attention gives it: context length + depth - 1
// (LLM Primer VI ch. 9 §9.2: a candidate tree is checked in one pass with positions by depth).
//
// Every element is read and written once: HBM bounds it.  D / 8 lanes hold a head's row, eight
// channels each, chosen so that both of a rotated pair are in the same lane; they share out the
// row's heads in groups, with the angles computed once per group.
//
// Angles: t / 2 pi = position * f, f = inv_freq / 2 pi.  Only the fraction of the turns counts,
// so f is held as a 64-bit fraction and the product is taken modulo 2^64: exact, whatever the
// position.  The nearest quarter turn is taken off before the rest (at most 1/8 turn) becomes
// a float.
#include <algorithm>

#include "tv_internal.cuh"

namespace tv {
namespace {

constexpr int kThreadsR = 256;
constexpr int kUnroll = 4;   // heads whose loads are in flight together
constexpr int kPerSm = 4;    // CTAs that registers leave room for

template <typename E>
struct Quad;
template <>
struct Quad<__nv_bfloat16> {
    uint2 w;
    __device__ void get(float (&x)[4]) const {
        x[0] = __uint_as_float(w.x << 16);
        x[1] = __uint_as_float(w.x & 0xFFFF0000u);
        x[2] = __uint_as_float(w.y << 16);
        x[3] = __uint_as_float(w.y & 0xFFFF0000u);
    }
    __device__ void set(const float (&x)[4]) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]),
                             b = __floats2bfloat162_rn(x[2], x[3]);
        w.x = *reinterpret_cast<const uint32_t *>(&a);
        w.y = *reinterpret_cast<const uint32_t *>(&b);
    }
};
template <>
struct Quad<float> {
    float4 w;
    __device__ void get(float (&x)[4]) const {
        x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
    }
    __device__ void set(const float (&x)[4]) { w = make_float4(x[0], x[1], x[2], x[3]); }
};

// Turns per position as a 64-bit fraction.
__device__ __forceinline__ uint64_t turns(double inv_freq) {
    double f = inv_freq * 0.15915494309189533577;  // 1 / 2 pi
    f -= floor(f);
    return (uint64_t)(f * 18446744073709551616.0);
}

// cos and sin of 2 pi position f.
__device__ __forceinline__ void turn(long long position, uint64_t f, float &c, float &s) {
    const uint64_t t = (uint64_t)position * f;
    const uint64_t quarter = (t + (1ull << 61)) >> 62;
    const int32_t rest = (int32_t)(int64_t)((t - (quarter << 62)) >> 32);  // in 2^-32 turns
    float s0, c0;
    sincospif((float)rest * 4.6566128730773926e-10f, &s0, &c0);
    const bool swap = quarter & 1;
    s = swap ? c0 : s0;
    c = swap ? s0 : c0;
    if (quarter & 2) s = -s;
    if ((quarter + 1) & 2) c = -c;
}

// Request of row `row`: the last one that begins at or before it, by a whole warp: a round of
// loads leaves a 32nd of the requests.
__device__ __forceinline__ int request_of(const int32_t *offs, int B, int row) {
    const int lane = threadIdx.x % 32;
    int lo = 0, n = B;
    while (n > 1) {
        const int each = (n + 31) / 32, at = lane * each;
        const uint32_t begun = __ballot_sync(0xffffffffu, at < n && offs[lo + at] <= row);
        const int skip = max(__popc(begun) - 1, 0) * each;
        lo += skip;
        n = min(each, n - skip);
    }
    return lo;
}

// 1 / sqrt(x): the hardware's and a step of Newton's method.
__device__ __forceinline__ float inv_sqrt(float x) {
    const float y = rsqrtf(x);
    return x < 3.0e38f ? y * fmaf(-0.5f * x * y, y, 1.5f) : y;
}

template <typename E, int D, bool PAIRS>
__global__ void __launch_bounds__(kThreadsR, sizeof(E) == 2 ? kPerSm : kPerSm / 2)
    qk_norm_rope_kernel(RopeArgs a, int per_item, int items_row) {
    constexpr int kLanes = D / 8;
    __shared__ uint64_t s_turns[D / 2];
    const int heads = a.H + a.Hkv;
    const int lane = threadIdx.x % 32, slot = threadIdx.x % kLanes;
    const long long items = (long long)a.R * items_row;
    const long long step = (long long)gridDim.x * (kThreadsR / kLanes);
    // channels of the lane's two quads
    const bool turned = slot < a.rot / 8;
    const int rest = slot - a.rot / 8;
    const int cA = PAIRS ? 8 * slot : turned ? 4 * slot : a.rot + 8 * rest;
    const int cB = PAIRS || !turned ? cA + 4 : a.rot / 2 + 4 * slot;
    using Q = Quad<E>;
    const bool norm = a.eps >= 0.f;
    pdl_wait();
    pdl_launch_next();
    // malformed offsets are told by one thread for each request
    for (long long b = (long long)blockIdx.x * kThreadsR + threadIdx.x; b < a.B;
         b += (long long)gridDim.x * kThreadsR) {
        int o, n;
        if (!request_range(a.offsets, (int)b, a.R, 0x7fffffff, o, n)) report(a.status, TV_ERR_TREE);
    }
    // up to 32 requests: their first rows and positions, one in each lane
    const int begins = lane < a.B ? a.offsets[lane] : 0x7fffffff;
    const int starts = lane < a.B ? a.start[lane] : 0;
    Q qA, qB, kA, kB;  // weights
    const float ones[4] = {1.f, 1.f, 1.f, 1.f};
    qA.set(ones);
    qB.set(ones);
    kA.set(ones);
    kB.set(ones);
    if (norm && a.q_weight) {
        qA = *reinterpret_cast<const Q *>(static_cast<const E *>(a.q_weight) + cA);
        qB = *reinterpret_cast<const Q *>(static_cast<const E *>(a.q_weight) + cB);
    }
    if (norm && a.k_weight && a.Hkv > 0) {
        kA = *reinterpret_cast<const Q *>(static_cast<const E *>(a.k_weight) + cA);
        kB = *reinterpret_cast<const Q *>(static_cast<const E *>(a.k_weight) + cB);
    }
    // a warp's first item, whose lanes' items follow it; every lane takes the same steps
    for (long long first = ((long long)blockIdx.x * kThreadsR + threadIdx.x - lane) / kLanes,
                   begin = first;
         first < items || begin == first; first += step) {
        const long long item = first + lane / kLanes;
        const bool there = item < items;
        const int row = there ? (int)(item / items_row) : 0;
        const int h0 = there ? (int)(item - (long long)row * items_row) * per_item : 0;
        const E *q = static_cast<const E *>(a.q) + (size_t)row * a.q_stride;
        const E *k = static_cast<const E *>(a.k) + (size_t)row * a.k_stride;
        const auto load = [&](int i, Q (&A)[kUnroll], Q (&B)[kUnroll]) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int h = h0 + i + u;
                const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                A[u].set(zero);
                B[u].set(zero);
                if (there && i + u < per_item && h < heads) {
                    const E *in = h < a.H ? q + h * D : k + (h - a.H) * D;
                    A[u] = *reinterpret_cast<const Q *>(in + cA);
                    B[u] = *reinterpret_cast<const Q *>(in + cB);
                }
            }
        };
        Q A[kUnroll], B[kUnroll];
        load(0, A, B);
        const int depth = a.depth && there ? a.depth[row] : 1;
        if (first == begin) {
            for (int i = threadIdx.x; i < a.rot / 2; i += kThreadsR)
                s_turns[i] = turns(a.inv_freq[i]);
            __syncthreads();
        }
        // the rows' requests and positions, a row of the warp after the other
        bool live = false;
        long long pos = 0;
#pragma unroll
        for (int g = 0; g < 32 / kLanes; ++g) {
            const int at = __shfl_sync(0xffffffffu, row, g * kLanes);
            const int b = a.B <= 32 ? max(__popc(__ballot_sync(0xffffffffu, begins <= at)) - 1, 0)
                                    : request_of(a.offsets, a.B, at);
            const int begin_row = a.offsets[b];
            const int p = a.B <= 32 ? __shfl_sync(0xffffffffu, starts, b) : a.start[b];
            int off, n;
            const bool in = request_range(a.offsets, b, a.R, 0x7fffffff, off, n) && at >= off &&
                            at < off + n;
            if (lane / kLanes == g) {
                live = there && in;
                pos = (long long)p + (a.depth ? depth - 1LL : at - begin_row);
            }
        }
        float cs[4], sn[4];
        if (turned) {
#pragma unroll
            for (int e = 0; e < 4; ++e) turn(pos, s_turns[4 * slot + e], cs[e], sn[e]);
        }
        E *q_out = static_cast<E *>(a.q_out) + (size_t)row * a.q_out_stride;
        E *k_out = static_cast<E *>(a.k_out) + (size_t)row * a.k_out_stride;
        for (int i = 0; i < per_item; i += kUnroll) {
            if (i > 0) load(i, A, B);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int h = h0 + i + u;
                const bool key = h >= a.H;
                float x[4], y[4];
                A[u].get(x);
                B[u].get(y);
                if (norm) {
                    float sum = 0.f, wA[4], wB[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum = fmaf(x[e], x[e], fmaf(y[e], y[e], sum));
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1)
                        sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    const float inv = inv_sqrt(fmaf(sum, 1.f / D, a.eps));
                    (key ? kA : qA).get(wA);
                    (key ? kB : qB).get(wB);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[e] = x[e] * inv * wA[e];
                        y[e] = y[e] * inv * wB[e];
                    }
                }
                if (turned) {
                    if (PAIRS) {
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const float x0 = x[e], y0 = y[e];
                            x[e] = x0 * cs[e / 2] - x[e + 1] * sn[e / 2];
                            x[e + 1] = x[e + 1] * cs[e / 2] + x0 * sn[e / 2];
                            y[e] = y0 * cs[2 + e / 2] - y[e + 1] * sn[2 + e / 2];
                            y[e + 1] = y[e + 1] * cs[2 + e / 2] + y0 * sn[2 + e / 2];
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float t = x[e] * cs[e] - y[e] * sn[e];
                            y[e] = y[e] * cs[e] + x[e] * sn[e];
                            x[e] = t;
                        }
                    }
                }
                if (live && i + u < per_item && h < heads) {
                    E *out = key ? k_out + (h - a.H) * D : q_out + h * D;
                    Q o;
                    o.set(x);
                    *reinterpret_cast<Q *>(out + cA) = o;
                    o.set(y);
                    *reinterpret_cast<Q *>(out + cB) = o;
                }
            }
        }
    }
}

template <typename E, int D, bool PAIRS>
cudaError_t launch(const RopeArgs &a, cudaStream_t s) {
    // Heads per item: about twenty where the rows alone fill the SMs, so that an angle serves many;
    // four where rows are few, so that their heads spread over the SMs.
    const long long heads = (long long)a.H + a.Hkv, lanes = device_sms() * 1024LL;
    const bool many = a.R * heads * (D / 8) >= 20 * lanes;
    long long items_row = many ? std::max(1LL, (heads + 10) / 20) : (heads + kUnroll - 1) / kUnroll;
    const int per_item = (int)(((heads + items_row - 1) / items_row + kUnroll - 1) / kUnroll * kUnroll);
    items_row = (heads + per_item - 1) / per_item;
    const int per_sm = sizeof(E) == 2 ? kPerSm : kPerSm / 2;
    const long long blocks = (a.R * items_row * (D / 8) + kThreadsR - 1) / kThreadsR;
    return launch_pdl(qk_norm_rope_kernel<E, D, PAIRS>,
                      dim3((unsigned)std::min(blocks, (long long)device_sms() * per_sm)),
                      dim3(kThreadsR), 0, s, a, per_item, (int)items_row);
}

template <typename E, int D>
cudaError_t launch(const RopeArgs &a, cudaStream_t s) {
    return a.pairs ? launch<E, D, true>(a, s) : launch<E, D, false>(a, s);
}

template <typename E>
cudaError_t launch(const RopeArgs &a, cudaStream_t s) {
    return a.d == 64 ? launch<E, 64>(a, s) : a.d == 128 ? launch<E, 128>(a, s) : launch<E, 256>(a, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs &a, cudaStream_t s) {
    return a.dtype == TV_BF16 ? launch<__nv_bfloat16>(a, s) : launch<float>(a, s);
}

}  // namespace tv
