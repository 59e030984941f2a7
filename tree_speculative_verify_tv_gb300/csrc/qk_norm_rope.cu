// qk_norm_rope.cu -- queries and keys of an attention layer normed per head and rotated at
// their positions, in one pass.
//
//   y_c = x_c w_c / sqrt(mean x^2 + eps);  (a, b) -> (a cos t - b sin t, b cos t + a sin t)
// A tree node stands at the position that tree attention gives it: context length + depth - 1
// (LLM Primer VI ch. 9 §9.2: a candidate tree is checked in one pass with positions by depth).
//
// Every element is read and written once: HBM bounds it, if the instructions stay few.  D / 8
// lanes hold a head's row, eight channels each, chosen so that both of a rotated pair are in the
// same lane; the lanes walk over heads of one row with weight * cos and weight * sin in
// registers, so a channel costs a multiply-add and a multiply of the packed kind beside its
// square and its conversions.
//
// Angles: t / 2 pi = position * f, f = inv_freq / 2 pi.  Only the fraction of the turns counts,
// so f is held as a 64-bit fraction and the product is taken modulo 2^64, which is exact.  f itself is
// a double's: off by 2^-52 of itself, so an angle of t rad by 2^-52 t (2^-21 at 2^31 rad; f as two
// doubles is better by that and takes 0.15 us more of a call of 4).  The nearest quarter turn is
// taken off before the rest (at most 1/8 turn) becomes a float.
#include <algorithm>
#include <type_traits>

#include "tv_internal.cuh"

namespace tv {
namespace {

constexpr int kThreadsR = 256;
constexpr int kUnroll = 4;   // heads whose loads are in flight together
// CTAs per SM that registers are kept to: three (80 registers a thread) for bf16, two for fp32.
// 32768 bf16 rows of 40 heads: 113 us, with four 121 (spills), with two 134.
template <typename E>
constexpr int kPerSm = sizeof(E) == 2 ? 3 : 2;

__device__ __forceinline__ Two swap(Two x) {
    const float2 y = halves(x);
    return two(y.y, y.x);
}

// Four channels as they lie in memory.
template <typename E>
struct Quad;
template <>
struct Quad<__nv_bfloat16> {
    uint2 w;
    __device__ void get(Two (&x)[2]) const {
        x[0] = two(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u));
        x[1] = two(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
    }
    __device__ void set(const Two (&x)[2]) {
        const __nv_bfloat162 a = __float22bfloat162_rn(halves(x[0])),
                             b = __float22bfloat162_rn(halves(x[1]));
        w.x = *reinterpret_cast<const uint32_t *>(&a);
        w.y = *reinterpret_cast<const uint32_t *>(&b);
    }
};
template <>
struct Quad<float> {
    float4 w;
    __device__ void get(Two (&x)[2]) const {
        x[0] = two(w.x, w.y);
        x[1] = two(w.z, w.w);
    }
    __device__ void set(const Two (&x)[2]) {
        const float2 a = halves(x[0]), b = halves(x[1]);
        w = make_float4(a.x, a.y, b.x, b.y);
    }
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

// Means of squares outside of these come from values whose squares, or their sum, may have left
// single precision.  Such a head's row is left out and done again, times a power of two.
constexpr float kLeast = 1.0e-30f, kMost = 3.0e38f;
constexpr float kShrink = 8.271806125530277e-25f, kGrow = 1.2676506002282294e30f;  // 2^-80, 2^100

// The sum of squares of a row of D channels, eight of them in this lane.
template <int D>
__device__ __forceinline__ float square_sum(const Two (&x)[2], const Two (&y)[2]) {
    const float2 q =
        halves(fma2(x[0], x[0], fma2(x[1], x[1], fma2(y[0], y[0], mul2(y[1], y[1])))));
    float sum = q.x + q.y;
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// A projection's weights with the rotation, for a lane's two quads (x: the first, y: the second).
struct Turned {
    Two xc[2], xs[2], yc[2], ys[2];
};

template <typename E, int D, bool PAIRS>
__global__ void __launch_bounds__(kThreadsR, kPerSm<E>)
    qk_norm_rope_kernel(RopeArgs a, int per_item, int items_row) {
    constexpr int kLanes = D / 8, kRowsWarp = 32 / kLanes;
    using Q = Quad<E>;
    __shared__ uint64_t s_turns[D / 2];
    const int heads = a.H + a.Hkv;
    const int lane = threadIdx.x % 32, slot = threadIdx.x % kLanes;
    // items: kRowsWarp rows and per_item heads, a warp each
    const long long rows_of = (a.R + kRowsWarp - 1LL) / kRowsWarp;
    const long long items = rows_of * items_row, step = (long long)gridDim.x * (kThreadsR / 32);
    const long long begin = (long long)blockIdx.x * (kThreadsR / 32) + threadIdx.x / 32;
    // channels of the lane's two quads
    const bool turned = slot < a.rot / 8;
    const int rest = slot - a.rot / 8;
    const int cA = PAIRS ? 8 * slot : turned ? 4 * slot : a.rot + 8 * rest;
    const int cB = PAIRS || !turned ? cA + 4 : a.rot / 2 + 4 * slot;
    const bool norm = a.eps >= 0.f;
    pdl_wait();
    pdl_launch_next();
    {  // the first item's first heads come nearer while angles and requests are looked up
        const int row = (int)min((begin / items_row) * kRowsWarp + lane / kLanes, a.R - 1LL);
        const int h = min((int)(begin % items_row) * per_item, a.H - 1);
        const E *x = static_cast<const E *>(a.q) + (size_t)row * a.q_stride + (size_t)h * D + cA;
        asm volatile("prefetch.global.L1 [%0];" ::"l"(x));
    }
    // malformed offsets are told by one thread for each request
    for (long long b = (long long)blockIdx.x * kThreadsR + threadIdx.x; b < a.B;
         b += (long long)gridDim.x * kThreadsR) {
        int o, n;
        if (!request_range(a.offsets, (int)b, a.R, 0x7fffffff, o, n)) report(a.status, TV_ERR_TREE);
    }
    // up to 32 requests: their first rows and positions, one in each lane
    const int begins = lane < a.B ? a.offsets[lane] : 0x7fffffff;
    const int starts = lane < a.B ? a.start[lane] : 0;
    for (int i = threadIdx.x; i < a.rot / 2; i += kThreadsR) s_turns[i] = turns(a.inv_freq[i]);
    __syncthreads();

    for (long long item = begin; item < items; item += step) {
        const long long rows = item / items_row;
        const int h0 = (int)(item - rows * items_row) * per_item, h1 = min(h0 + per_item, heads);
        const long long mine = rows * kRowsWarp + lane / kLanes;
        const int row = (int)min(mine, a.R - 1LL);
        const int depth = a.depth ? a.depth[row] : 1;
        // the rows' requests and positions, a row of the warp after the other
        bool live = false;
        long long pos = 0;
#pragma unroll
        for (int g = 0; g < kRowsWarp; ++g) {
            const int at = __shfl_sync(0xffffffffu, row, g * kLanes);
            const int b = a.B <= 32 ? max(__popc(__ballot_sync(0xffffffffu, begins <= at)) - 1, 0)
                                    : request_of(a.offsets, a.B, at);
            const int p = a.B <= 32 ? __shfl_sync(0xffffffffu, starts, b) : a.start[b];
            int off, n;
            const bool in = request_range(a.offsets, b, a.R, 0x7fffffff, off, n) && at >= off &&
                            at < off + n;
            if (lane / kLanes == g) {
                live = mine < a.R && in;
                pos = (long long)p + (a.depth ? depth - 1LL : at - off);
            }
        }
        float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
        if (turned) {
#pragma unroll
            for (int e = 0; e < 4; ++e) turn(pos, s_turns[4 * slot + e], cs[e], sn[e]);
        }
        // `n` heads of one projection
        const auto project = [&](const E *in, E *out, int n, const E *weight) {
            Two wx[2] = {two(1.f, 1.f), two(1.f, 1.f)}, wy[2] = {wx[0], wx[0]};
            if (norm && weight) {
                reinterpret_cast<const Q *>(weight + cA)->get(wx);
                reinterpret_cast<const Q *>(weight + cB)->get(wy);
            }
            // HALVES: x' = x wx cos - y wy sin, y' = y wy cos + x wx sin.
            // PAIRS: (a, b)' = (a, b) w (cos, cos) + (b, a) w' (-sin, sin), within x and within y.
            Turned f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (PAIRS) {
                    f.xc[e] = mul2(wx[e], two(cs[e], cs[e]));
                    f.yc[e] = mul2(wy[e], two(cs[2 + e], cs[2 + e]));
                    f.xs[e] = mul2(swap(wx[e]), two(-sn[e], sn[e]));
                    f.ys[e] = mul2(swap(wy[e]), two(-sn[2 + e], sn[2 + e]));
                } else {
                    const Two c = two(cs[2 * e], cs[2 * e + 1]), s = two(sn[2 * e], sn[2 * e + 1]);
                    f.xc[e] = mul2(wx[e], c);
                    f.yc[e] = mul2(wy[e], c);
                    f.xs[e] = mul2(wx[e], s);
                    f.ys[e] = mul2(wy[e], two(-sn[2 * e], -sn[2 * e + 1]));
                }
            }
            in += cA;
            out += cA;
            const int over = cB - cA;
            // a normed row rotated and stored
            const auto put = [&](Two (&x)[2], Two (&y)[2], E *to) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const Two p = x[e], r = y[e];
                    if (!turned) {
                        x[e] = mul2(p, f.xc[e]);
                        y[e] = mul2(r, f.yc[e]);
                    } else if (PAIRS) {
                        x[e] = fma2(p, f.xc[e], mul2(swap(p), f.xs[e]));
                        y[e] = fma2(r, f.yc[e], mul2(swap(r), f.ys[e]));
                    } else {
                        x[e] = fma2(p, f.xc[e], mul2(r, f.ys[e]));
                        y[e] = fma2(r, f.yc[e], mul2(p, f.xs[e]));
                    }
                }
                Q o;
                o.set(x);
                *reinterpret_cast<Q *>(to) = o;
                o.set(y);
                *reinterpret_cast<Q *>(to + over) = o;
            };
            uint32_t again = 0;  // heads (fewer than 32 in an item) left out
            const auto some = [&](auto count, int h) {
                constexpr int kCount = decltype(count)::value;
                Q A[kCount], B[kCount];
#pragma unroll
                for (int u = 0; u < kCount; ++u) {
                    A[u] = *reinterpret_cast<const Q *>(in + (h + u) * D);
                    B[u] = *reinterpret_cast<const Q *>(in + (h + u) * D + over);
                }
#pragma unroll
                for (int u = 0; u < kCount; ++u) {
                    Two x[2], y[2];
                    A[u].get(x);
                    B[u].get(y);
                    bool fits = true;
                    if (norm) {
                        const float mean = fmaf(square_sum<D>(x, y), 1.f / D, a.eps);
                        fits = mean >= kLeast && mean <= kMost;
                        if (!fits) again |= 1u << (h + u);
                        const float i = inv_sqrt(mean);
                        const Two inv = two(i, i);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            x[e] = mul2(x[e], inv);
                            y[e] = mul2(y[e], inv);
                        }
                    }
                    if (live && fits) put(x, y, out + (h + u) * D);
                }
            };
            int h = 0;
#pragma unroll 1
            for (; h + kUnroll <= n; h += kUnroll) some(std::integral_constant<int, kUnroll>(), h);
#pragma unroll 1
            for (; h < n; ++h) some(std::integral_constant<int, 1>(), h);
            // (rows of one warp may differ in what is left; in place, what is done is not read again)
            for (uint32_t rest = __reduce_or_sync(0xffffffffu, again); rest; rest &= rest - 1) {
                const int at = __ffs(rest) - 1;
                Two x[2], y[2];
                reinterpret_cast<const Q *>(in + at * D)->get(x);
                reinterpret_cast<const Q *>(in + at * D + over)->get(y);
                const float mean = fmaf(square_sum<D>(x, y), 1.f / D, a.eps);
                const float scale = mean < kLeast ? kGrow : kShrink;
                const Two s2 = two(scale, scale);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    x[e] = mul2(x[e], s2);
                    y[e] = mul2(y[e], s2);
                }
                const float i = inv_sqrt(fmaf(square_sum<D>(x, y), 1.f / D, a.eps * scale * scale));
                const Two inv = two(i, i);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    x[e] = mul2(x[e], inv);
                    y[e] = mul2(y[e], inv);
                }
                if (live && (again >> at & 1)) put(x, y, out + at * D);
            }
        };
        if (h0 < a.H)
            project(static_cast<const E *>(a.q) + (size_t)row * a.q_stride + (size_t)h0 * D,
                    static_cast<E *>(a.q_out) + (size_t)row * a.q_out_stride + (size_t)h0 * D,
                    min(h1, a.H) - h0, static_cast<const E *>(a.q_weight));
        if (h1 > a.H) {
            const int from = max(h0, a.H);
            project(static_cast<const E *>(a.k) + (size_t)row * a.k_stride + (size_t)(from - a.H) * D,
                    static_cast<E *>(a.k_out) + (size_t)row * a.k_out_stride +
                        (size_t)(from - a.H) * D,
                    h1 - from, static_cast<const E *>(a.k_weight));
        }
    }
}

template <typename E, int D, bool PAIRS>
cudaError_t launch(const RopeArgs &a, cudaStream_t s) {
    // Heads per item: about twenty where the rows alone fill the SMs twice, so that an angle serves
    // many; down to four where rows are few, so that their heads spread over the SMs.  29 at most: the
    // kernel has a bit for each.
    const long long heads = (long long)a.H + a.Hkv, warps = kThreadsR / 32;
    const long long rows = (a.R + 256 / D - 1LL) / (256 / D);
    const long long resident = device_sms() * kPerSm<E> * warps;
    long long items_row = std::max((2 * resident + rows - 1) / rows, std::max(1LL, (heads + 10) / 20));
    items_row = std::min(items_row, (heads + kUnroll - 1) / kUnroll);
    const int per_item = (int)(((heads + items_row - 1) / items_row + kUnroll - 1) / kUnroll * kUnroll);
    items_row = (heads + per_item - 1) / per_item;
    const long long blocks = std::min((rows * items_row + warps - 1) / warps, resident / warps);
    return launch_pdl(qk_norm_rope_kernel<E, D, PAIRS>,
                      dim3((unsigned)blocks), dim3(kThreadsR), 0, s, a, per_item, (int)items_row);
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
