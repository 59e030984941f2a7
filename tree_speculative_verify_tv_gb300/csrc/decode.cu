// decode.cu -- one token of every request through the gated linear recurrence.
//
//   H' = diag(e^g) H + k v^T,   out = H'^T q   (Bole summary page, "Core techniques" §1, one step)
//
// The state is read and written once, 8 bytes an element against 5 operations: HBM bounds it (128
// requests of 32 heads, 128 x 128: 80 us, 6.7 TB/s).
// The decay is a pair of floats, as it is for prompts: one near 1, rounded to a float and applied
// token after token, would be off in the same direction every time (e^-1e-5 over 40000 tokens:
// 3e-4 of the state).
// A CTA takes columns of one (request, head): a thread holds a float4 of columns and walks down
// the key rows, kItems of its loads in flight; the read-out's partial sums of the row groups
// meet in shared memory.
#include "recurrence.cuh"

namespace tv {
namespace {

constexpr int kThreadsD = 256;
constexpr int kItems = 8;    // float4s of the state per thread and round
constexpr int kPerSmD = 4;   // CTAs per SM; with 16 items and two: 90 us for those 128 requests

template <typename E, bool DIAG>
__global__ void __launch_bounds__(kThreadsD, kPerSmD) decode_kernel(DecodeArgs a, int cols) {
    __shared__ float s_k[kMaxDim], s_q[kMaxDim];
    __shared__ rec::Pair s_d[DIAG ? kMaxDim : 1];
    __shared__ float4 s_sum[kThreadsD];
    const int unit = blockIdx.x, b = unit / a.H, h = unit % a.H, tid = threadIdx.x;
    const int c0 = blockIdx.y * cols, quads = min(cols, a.dv - c0) / 4;
    const int groups = kThreadsD / quads, group = tid / quads, quad = tid % quads;
    pdl_wait();
    pdl_launch_next();
    if (a.active && a.active[b] == 0) return;
    const size_t at = (size_t)unit * a.dk * a.dv + c0 + quad * 4;
    const float *H0 = a.H0 + at;
    float *H1 = a.H_new + at;
    const bool live = group < groups;

    // (what the decay comes from ahead of the state: its exponential is done before that is there)
    static_assert(kMaxDim <= kThreadsD, "a channel per thread");
    const float *g = a.g + (size_t)b * a.g_stride + (size_t)h * (DIAG ? a.dk : 1);
    const bool channel = tid < a.dk;
    const float gate = !DIAG ? g[0] : channel ? g[tid] : 0.f;
    float4 x[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int r = group + i * groups;
        if (live && r < a.dk) x[i] = rec::load4(H0 + (size_t)r * a.dv);
    }
    const E *k = static_cast<const E *>(a.k) + (size_t)b * a.k_stride + (size_t)h * a.dk;
    const E *q = static_cast<const E *>(a.q) + (size_t)b * a.q_stride + (size_t)h * a.dk;
    const E *v = static_cast<const E *>(a.v) + (size_t)b * a.v_stride + (size_t)h * a.dv + c0;
    const float4 v4 = rec::load4(v + quad * 4);
    const rec::Pair d = rec::exp_pair(gate);
    if (channel) {
        s_k[tid] = to_f32(k[tid]);
        s_q[tid] = to_f32(q[tid]);
        if (DIAG) s_d[tid] = d;
    }
    __syncthreads();

    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int base = 0; base < a.dk; base += kItems * groups) {
        if (base > 0) {
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const int r = base + group + i * groups;
                if (live && r < a.dk) x[i] = rec::load4(H0 + (size_t)r * a.dv);
            }
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int r = base + group + i * groups;
            if (live && r < a.dk) {
                const float kr = s_k[r], qr = s_q[r];
                const rec::Pair dr = DIAG ? s_d[r] : d;
                float4 y;
                y.x = fmaf(x[i].x, dr.hi, fmaf(x[i].x, dr.lo, kr * v4.x));
                y.y = fmaf(x[i].y, dr.hi, fmaf(x[i].y, dr.lo, kr * v4.y));
                y.z = fmaf(x[i].z, dr.hi, fmaf(x[i].z, dr.lo, kr * v4.z));
                y.w = fmaf(x[i].w, dr.hi, fmaf(x[i].w, dr.lo, kr * v4.w));
                *reinterpret_cast<float4 *>(H1 + (size_t)r * a.dv) = y;
                o.x = fmaf(y.x, qr, o.x);
                o.y = fmaf(y.y, qr, o.y);
                o.z = fmaf(y.z, qr, o.z);
                o.w = fmaf(y.w, qr, o.w);
            }
        }
    }
    s_sum[tid] = o;
    __syncthreads();
    const float *sums = reinterpret_cast<const float *>(s_sum);
    for (int c = tid; c < quads * 4; c += kThreadsD) {
        float t = 0.f;
        for (int j = 0; j < groups; ++j) t += sums[j * quads * 4 + c];
        rec::store_out(a.out, a.out_f32, (size_t)unit * a.dv + c0 + c, t);
    }
}

template <typename E, bool DIAG>
cudaError_t launch(const DecodeArgs &a, cudaStream_t s) {
    // columns per CTA: all of a head's, or pieces of 32 (128-byte rows) where the heads alone
    // leave SMs without work
    const int sms = device_sms(), units = a.B * a.H;
    const int cols = units < 2 * sms ? 32 : a.dv;
    return launch_pdl(decode_kernel<E, DIAG>,
                      dim3((unsigned)units, (unsigned)((a.dv + cols - 1) / cols)),
                      dim3(kThreadsD), 0, s, a, cols);
}

}  // namespace

cudaError_t launch_decode(const DecodeArgs &a, cudaStream_t s) {
    const bool diag = a.decay == TV_DECAY_DIAG;
    if (a.qkv_dtype == TV_BF16)
        return diag ? launch<__nv_bfloat16, true>(a, s) : launch<__nv_bfloat16, false>(a, s);
    return diag ? launch<float, true>(a, s) : launch<float, false>(a, s);
}

}  // namespace tv
