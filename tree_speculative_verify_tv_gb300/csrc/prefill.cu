// prefill.cu -- prompts through the gated linear recurrence, row by row on CUDA cores, and the
// choice between this kernel and the tensor-core one.
//
//   H_t = diag(e^{g_t}) H_{t-1} + k_t v_t^T,   out_t = H_t^T q_t
// (Bole summary page, "Core techniques" §1: h_{t+1} = S_t h_t + u_t)
//
// A CTA takes 16 columns of one (request, head) and walks down the rows.  Eight lanes share a
// column, each with 4 ceil(dk / 32) rows of the state in registers; blocks of kRows rows of
// q, k, v land in shared memory by asynchronous copies a block ahead.  A pair of the state takes
// four packed instructions (one for the decay's second part) against dk-sized loads: instructions
// bound it.  8000 fp32 rows of 24 heads, 128 x 128: 727 us with two columns a thread, 64 x 64: 260;
// with a decay per channel 1375.
#include "recurrence.cuh"
#include "tc_ptx.cuh"

namespace tv {
namespace {

constexpr int kThreadsP = 128;
constexpr int kCols = 16;  // columns per CTA, one or two times
constexpr int kRows = 8;   // rows per block of copies

template <typename E, bool DIAG, int R, int N>
struct RowsSmem {
    E k[2][kRows][32 * R], q[2][kRows][32 * R], v[2][kRows][N * kCols];
    rec::Pair d[2][kRows][DIAG ? 32 * R : 1];
};

// R: groups of 32 key rows; N: columns of a thread.
template <typename E, bool DIAG, int R, int N>
__global__ void __launch_bounds__(kThreadsP) prefill_rows_kernel(PrefillArgs a) {
    extern __shared__ __align__(16) uint8_t s_raw[];
    auto &s = *reinterpret_cast<RowsSmem<E, DIAG, R, N> *>(s_raw);
    constexpr int kPiece = 16 / sizeof(E);  // elements per copy
    const int unit = blockIdx.x, b = unit / a.H, h = unit % a.H, tid = threadIdx.x;
    const int c0 = blockIdx.y * N * kCols, cols = min(N * kCols, a.dv - c0);
    const int r = tid % 8, col = tid / 8;
    pdl_wait();
    pdl_launch_next();
    int off, n;
    if (!request_range(a.offsets, b, a.R, a.max_rows, off, n)) {
        if (tid == 0) report(a.status, TV_ERR_TREE);
        return;
    }
    // channels past dk stay zero in both buffers
    for (int i = tid; i < 2 * kRows * (32 * R - a.dk); i += kThreadsP) {
        const int c = a.dk + i % (32 * R - a.dk), t = i / (32 * R - a.dk);
        s.k[t / kRows][t % kRows][c] = E(0.f);
        s.q[t / kRows][t % kRows][c] = E(0.f);
        if (DIAG) s.d[t / kRows][t % kRows][c] = {0.f, 0.f};
    }
    const size_t state = (size_t)unit * a.dk * a.dv + c0 + col;
    Two x[N][2 * R];  // pairs of rows
#pragma unroll
    for (int w = 0; w < N; ++w)
#pragma unroll
        for (int i = 0; i < 2 * R; ++i) {
            const int row = (i / 2) * 32 + 4 * r + i % 2 * 2;  // (dk is even)
            const bool have = a.H0 && col + w * kCols < cols && row < a.dk;
            const float *from = a.H0 + state + w * kCols;
            x[w][i] = have ? two(from[(size_t)row * a.dv], from[(size_t)(row + 1) * a.dv]) : 0;
        }

    constexpr int kGates = DIAG ? kRows * 32 * R / kThreadsP : 1;
    float gates[kGates];
    const auto fetch = [&](int t0, int buf) {  // rows t0 .. of the request into a buffer
        const int cnt = min(kRows, n - t0), pk = a.dk / kPiece, pv = cols / kPiece;
        for (int i = tid; i < cnt * pk; i += kThreadsP) {
            const int t = i / pk, c = i % pk * kPiece;
            const size_t row = (size_t)off + t0 + t;
            ptx::cp_async_16(ptx::smem_addr(&s.k[buf][t][c]),
                             static_cast<const E *>(a.k) + row * a.k_stride + (size_t)h * a.dk + c);
            ptx::cp_async_16(ptx::smem_addr(&s.q[buf][t][c]),
                             static_cast<const E *>(a.q) + row * a.q_stride + (size_t)h * a.dk + c);
        }
        for (int i = tid; i < cnt * pv; i += kThreadsP) {
            const int t = i / pv, c = i % pv * kPiece;
            ptx::cp_async_16(ptx::smem_addr(&s.v[buf][t][c]),
                             static_cast<const E *>(a.v) + ((size_t)off + t0 + t) * a.v_stride +
                                 (size_t)h * a.dv + c0 + c);
        }
#pragma unroll
        for (int j = 0; j < kGates; ++j) {
            const int i = tid + j * kThreadsP, t = DIAG ? i / a.dk : i, c = DIAG ? i % a.dk : 0;
            gates[j] = t < cnt ? a.g[((size_t)off + t0 + t) * a.g_stride +
                                     (size_t)h * (DIAG ? a.dk : 1) + c]
                               : 0.f;
        }
    };
    if (n > 0) fetch(0, 0);
    for (int t0 = 0, buf = 0; t0 < n; t0 += kRows, buf ^= 1) {
        const int cnt = min(kRows, n - t0);
#pragma unroll
        for (int j = 0; j < kGates; ++j) {
            const int i = tid + j * kThreadsP, t = DIAG ? i / a.dk : i, c = DIAG ? i % a.dk : 0;
            if (t < kRows) s.d[buf][t][c] = rec::exp_pair(gates[j]);
        }
        ptx::cp_async_wait_all();
        __syncthreads();
        if (t0 + kRows < n) fetch(t0 + kRows, buf ^ 1);
        float mine[N] = {};
#pragma unroll 2
        for (int t = 0; t < cnt; ++t) {
            const rec::Pair d = s.d[buf][t][0];
            Two v2[N], hi = two(d.hi, d.hi), lo = two(d.lo, d.lo), o2[N] = {};
#pragma unroll
            for (int w = 0; w < N; ++w) {
                const float vc = to_f32(s.v[buf][t][col + w * kCols]);
                v2[w] = two(vc, vc);
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int c = i * 32 + 4 * r;
                const float4 k4 = rec::load4(&s.k[buf][t][c]), q4 = rec::load4(&s.q[buf][t][c]);
                const Two kk[2] = {two(k4.x, k4.y), two(k4.z, k4.w)};
                const Two qq[2] = {two(q4.x, q4.y), two(q4.z, q4.w)};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (DIAG) {
                        const rec::Pair d0 = s.d[buf][t][c + 2 * e], d1 = s.d[buf][t][c + 2 * e + 1];
                        hi = two(d0.hi, d1.hi);
                        lo = two(d0.lo, d1.lo);
                    }
#pragma unroll
                    for (int w = 0; w < N; ++w) {
                        Two &y = x[w][2 * i + e];
                        y = fma2(y, hi, fma2(y, lo, mul2(kk[e], v2[w])));
                        o2[w] = fma2(y, qq[e], o2[w]);
                    }
                }
            }
#pragma unroll
            for (int w = 0; w < N; ++w) {
                const float2 os = halves(o2[w]);
                float o = os.x + os.y;
                o += __shfl_xor_sync(0xffffffffu, o, 1);
                o += __shfl_xor_sync(0xffffffffu, o, 2);
                o += __shfl_xor_sync(0xffffffffu, o, 4);
                if (t == r) mine[w] = o;
            }
        }
#pragma unroll
        for (int w = 0; w < N; ++w)
            if (col + w * kCols < cols && r < cnt)
                rec::store_out(a.out, a.out_f32,
                               (((size_t)off + t0 + r) * a.H + h) * a.dv + c0 + col + w * kCols,
                               mine[w]);
    }
#pragma unroll
    for (int w = 0; w < N; ++w)
#pragma unroll
        for (int i = 0; i < 2 * R; ++i) {
            const int row = (i / 2) * 32 + 4 * r + i % 2 * 2;
            const float2 y = halves(x[w][i]);
            float *to = a.H_new + state + w * kCols;
            if (col + w * kCols < cols && row < a.dk) {
                to[(size_t)row * a.dv] = y.x;
                to[(size_t)(row + 1) * a.dv] = y.y;
            }
        }
}

constexpr int kTwo = 2;  // CTAs per SM that two columns a thread have to leave

template <typename E, bool DIAG, int R, int N>
cudaError_t launch_columns(const PrefillArgs &a, cudaStream_t s) {
    const cudaError_t e = configure_smem_once(prefill_rows_kernel<E, DIAG, R, N>, false);
    if (e != cudaSuccess) return e;
    return launch_pdl(prefill_rows_kernel<E, DIAG, R, N>,
                      dim3((unsigned)(a.B * a.H), (unsigned)((a.dv + N * kCols - 1) / (N * kCols))),
                      dim3(kThreadsP), sizeof(RowsSmem<E, DIAG, R, N>), s, a);
}

template <typename E, bool DIAG, int R>
cudaError_t launch_rows(const PrefillArgs &a, cudaStream_t s) {
    // Two columns a thread halve the loads of q and k per column, where that leaves enough CTAs.
    const bool two = (long long)a.B * a.H * ((a.dv + 2 * kCols - 1) / (2 * kCols)) >= kTwo * device_sms();
    return two ? launch_columns<E, DIAG, R, 2>(a, s) : launch_columns<E, DIAG, R, 1>(a, s);
}

template <typename E, bool DIAG>
cudaError_t launch_rows(const PrefillArgs &a, cudaStream_t s) {
    if (a.dk <= 32) return launch_rows<E, DIAG, 1>(a, s);
    if (a.dk <= 64) return launch_rows<E, DIAG, 2>(a, s);
    if (a.dk <= 128) return launch_rows<E, DIAG, 4>(a, s);
    return launch_rows<E, DIAG, 8>(a, s);
}

}  // namespace

bool prefill_fits(const PrefillArgs &a) {
    return a.R <= 0x7fff0000;  // rows, and a chunk behind them, are counted in 32 bits
}

size_t prefill_workspace_bytes(const PrefillArgs &a) {
    return a.B > 0 && prefill_tc_supported(a) ? prefill_tc_workspace_bytes(a) : 0;
}

cudaError_t launch_prefill(const PrefillArgs &a, bool expire, cudaStream_t s) {
    if (prefill_tc_supported(a)) return launch_prefill_tc(a, expire, s);
    const bool diag = a.decay == TV_DECAY_DIAG;
    if (a.qkv_dtype == TV_BF16)
        return diag ? launch_rows<__nv_bfloat16, true>(a, s)
                    : launch_rows<__nv_bfloat16, false>(a, s);
    return diag ? launch_rows<float, true>(a, s) : launch_rows<float, false>(a, s);
}

}  // namespace tv
