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
#include "tv_internal.cuh"

namespace tv {
namespace {

constexpr int kThreadsR = 256;
constexpr int kUnroll = 4;  // heads whose loads are in flight together

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

// cos and sin of 2 pi position f.
__device__ __forceinline__ void turn(long long position, double inv_freq, float &c, float &s) {
    double f = inv_freq * 0.15915494309189533577;  // turns per position
    f -= floor(f);
    const uint64_t part = (uint64_t)(f * 18446744073709551616.0);
    const uint64_t t = (uint64_t)position * part;
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

// Request of row `row`: the last one that begins at or before it.
__device__ __forceinline__ int request_of(const int32_t *offs, int B, int row) {
    int lo = 0, n = B;
    while (n > 1) {
        const int half = n / 2;
        if (offs[lo + half] <= row) {
            lo += half;
            n -= half;
        } else {
            n = half;
        }
    }
    return lo;
}

template <typename E, int D, bool PAIRS>
__global__ void __launch_bounds__(kThreadsR) qk_norm_rope_kernel(RopeArgs a, int per_item) {
    constexpr int kLanes = D / 8;
    const int heads = a.H + a.Hkv, items_row = (heads + per_item - 1) / per_item;
    const int slot = threadIdx.x % kLanes;
    const long long item =
        ((long long)blockIdx.x * kThreadsR + threadIdx.x) / kLanes;
    const int row = (int)min(item / items_row, (long long)a.R);
    const int h0 = (int)(item % items_row) * per_item, h1 = min(h0 + per_item, heads);
    pdl_wait();
    pdl_launch_next();
    // malformed offsets are told by the threads of the first items, one request each
    for (long long b = (long long)blockIdx.x * kThreadsR + threadIdx.x; b < a.B;
         b += (long long)gridDim.x * kThreadsR) {
        int o, n;
        if (!request_range(a.offsets, (int)b, a.R, 0x7fffffff, o, n)) report(a.status, TV_ERR_TREE);
    }
    bool live = row < a.R;
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    // channels of the lane's two quads
    const bool turned = slot < a.rot / 8;
    const int rest = slot - a.rot / 8;
    const int cA = PAIRS ? 8 * slot : turned ? 4 * slot : a.rot + 8 * rest;
    const int cB = PAIRS || !turned ? cA + 4 : a.rot / 2 + 4 * slot;
    if (live) {
        const int b = request_of(a.offsets, a.B, row);
        int off, n;
        live = request_range(a.offsets, b, a.R, 0x7fffffff, off, n) && row >= off && row < off + n;
        if (live && turned) {
            const long long pos = (long long)a.start[b] + (a.depth ? a.depth[row] - 1LL : row - off);
#pragma unroll
            for (int e = 0; e < 4; ++e) turn(pos, a.inv_freq[4 * slot + e], cs[e], sn[e]);
        }
    }
    using Q = Quad<E>;
    const bool norm = a.eps >= 0.f;
    float w[2][8];  // weights of queries and keys
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const E *weight = static_cast<const E *>(p ? a.k_weight : a.q_weight);
        float x[4] = {1.f, 1.f, 1.f, 1.f}, y[4] = {1.f, 1.f, 1.f, 1.f};
        if (norm && weight && (p == 0 || a.Hkv > 0)) {
            reinterpret_cast<const Q *>(weight + cA)->get(x);
            reinterpret_cast<const Q *>(weight + cB)->get(y);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[p][e] = x[e];
            w[p][4 + e] = y[e];
        }
    }
    const size_t at = live ? row : 0;
    const E *q = static_cast<const E *>(a.q) + at * a.q_stride;
    const E *k = static_cast<const E *>(a.k) + at * a.k_stride;
    E *q_out = static_cast<E *>(a.q_out) + at * a.q_out_stride;
    E *k_out = static_cast<E *>(a.k_out) + at * a.k_out_stride;
    // (every lane takes the same steps, whatever its row: the sums are shuffled)
    for (int i = 0; i < per_item; i += kUnroll) {
        Q rawA[kUnroll], rawB[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = h0 + i + u;
            const float zero[4] = {0.f, 0.f, 0.f, 0.f};
            rawA[u].set(zero);
            rawB[u].set(zero);
            if (live && i + u < per_item && h < heads) {
                const E *in = h < a.H ? q + (size_t)h * D : k + (size_t)(h - a.H) * D;
                rawA[u] = *reinterpret_cast<const Q *>(in + cA);
                rawB[u] = *reinterpret_cast<const Q *>(in + cB);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = h0 + i + u;
            const bool key = h >= a.H;
            float x[4], y[4];
            rawA[u].get(x);
            rawB[u].get(y);
            if (norm) {
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) sum = fmaf(x[e], x[e], fmaf(y[e], y[e], sum));
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const float inv = 1.f / sqrtf(sum * (1.f / D) + a.eps);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = x[e] * inv * (key ? w[1][e] : w[0][e]);
                    y[e] = y[e] * inv * (key ? w[1][4 + e] : w[0][4 + e]);
                }
            }
            if (turned) {
                if (PAIRS) {
                    const float z[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
                    float t[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        t[2 * e] = z[2 * e] * cs[e] - z[2 * e + 1] * sn[e];
                        t[2 * e + 1] = z[2 * e + 1] * cs[e] + z[2 * e] * sn[e];
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[e] = t[e];
                        y[e] = t[4 + e];
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
                E *out = key ? k_out + (size_t)(h - a.H) * D : q_out + (size_t)h * D;
                Q o;
                o.set(x);
                *reinterpret_cast<Q *>(out + cA) = o;
                o.set(y);
                *reinterpret_cast<Q *>(out + cB) = o;
            }
        }
    }
}

template <typename E, int D, bool PAIRS>
cudaError_t launch(const RopeArgs &a, cudaStream_t s) {
    // heads per item: many rows share an angle among sixteen heads; few rows spread their heads
    // over the SMs
    const long long heads = (long long)a.H + a.Hkv, rows_wave = device_sms() * 2048LL / (D / 8);
    const int per_item = a.R * heads >= 16 * rows_wave ? 16 : kUnroll;
    const long long threads = a.R * ((heads + per_item - 1) / per_item) * (D / 8);
    const long long blocks = (threads + kThreadsR - 1) / kThreadsR;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_pdl(qk_norm_rope_kernel<E, D, PAIRS>, dim3((unsigned)blocks), dim3(kThreadsR), 0,
                      s, a, per_item);
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
