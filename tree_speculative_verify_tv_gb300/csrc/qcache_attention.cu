// qcache_attention.cu -- tree-masked softmax attention over the paged 4-bit KV cache.
//
// Query row (node i, head h) of request b sees the cached positions below ctx_len[b] and
// the nodes of i's root path, within the window or among the sinks:
//   o = sum_j softmax_j(scale * q . k_j) v_j.
// One CTA per query row: keys in tiles of 64 (a page, or 64 nodes of the root path), one
// thread per key for the scores, one per channel for the value sums, the running maximum
// and sum in fp32.
#include "qcache.cuh"

namespace tv {
namespace {

__device__ __forceinline__ float block_max(float x, float *s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    __syncthreads();
    if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = x;
    __syncthreads();
    return fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
}

template <int D>
__global__ void __launch_bounds__(128) qcache_attention_kernel(const QAttnArgs a) {
    using R = qc::Rec<D>;
    __shared__ float s_q[D], s_p[64], s_red[4];
    __shared__ int s_path[kMaxNodes];
    __shared__ int s_len, s_bad;
    const int tid = threadIdx.x;
    const int b = blockIdx.x / a.max_nodes, i = blockIdx.x % a.max_nodes, h = blockIdx.y;
    const int kvh = h / (a.H / a.Hkv);
    pdl_wait();
    pdl_launch_next();
    int off, n;
    const bool range = request_range(a.node_offsets, b, a.T, a.max_nodes, off, n);
    if (!range && tid == 0) report(a.status, TV_ERR_TREE);
    if (!range || i >= n) return;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    for (int t = tid; t < n; t += 128) {
        const int p = a.parent[off + t];
        if (p < -1 || p >= t) s_bad = TV_ERR_TREE;
    }
    __syncthreads();
    const int ctx = a.ctx_len[b];
    if (tid == 0 && !s_bad && (ctx < 0 || ctx > (long long)a.max_pages * kQPage))
        s_bad = TV_ERR_SHAPE;
    if (tid == 0 && !s_bad) {
        int len = 0;
        for (int t = i; t >= 0; t = a.parent[off + t]) s_path[len++] = t;
        s_len = len;
    }
    __syncthreads();
    const int sinks = a.window > 0 ? min(a.sinks, max(ctx, 0)) : 0;
    const int depth = s_len;
    // the window's first position for this node, and for any node of the request
    const long long lo = a.window > 0 ? max(0LL, (long long)ctx + depth - a.window) : 0;
    const long long lo1 = a.window > 0 ? max(0LL, (long long)ctx + 1 - a.window) : 0;
    if (!s_bad)
        for (int p = tid; p * kQPage < ctx; p += 128) {
            if (p * kQPage >= sinks && (p + 1LL) * kQPage <= lo1) continue;
            const int page = a.table[(size_t)b * a.max_pages + p];
            if (page < 0 || page >= a.num_pages) s_bad = TV_ERR_SHAPE;
        }
    __syncthreads();
    const size_t row = (size_t)(off + i) * a.H + h;
    float *of = static_cast<float *>(a.out) + row * D;
    __nv_bfloat16 *oh = static_cast<__nv_bfloat16 *>(a.out) + row * D;
    if (s_bad) {
        if (tid == 0) report(a.status, s_bad);
        if (tid < D) {
            if (a.out_f32)
                of[tid] = 0.f;
            else
                oh[tid] = __float2bfloat16_rn(0.f);
        }
        return;
    }
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q);
    if (tid < D) s_q[tid] = __bfloat162float(q[(size_t)(off + i) * a.q_stride + h * D + tid]);
    __syncthreads();
    const float ninf = __uint_as_float(0xff800000u);
    float m = ninf, l = 0.f, o = 0.f;
    const int pages = (ctx + kQPage - 1) / kQPage, tiles = pages + (depth + 63) / 64;
    for (int t = 0; t < tiles; ++t) {
        if (t < pages && t * kQPage >= sinks && (t + 1LL) * kQPage <= lo) continue;
        const uint8_t *rec = nullptr;
        if (t < pages)
            rec = a.cache +
                  ((size_t)a.table[(size_t)b * a.max_pages + t] * a.Hkv + kvh) * R::kBytes;
        float x = ninf;
        if (tid < 64 && t < pages) {
            const int pos = t * kQPage + tid;
            if (pos < ctx && (pos >= lo || pos < sinks)) {
                x = 0.f;
                for (int g = 0; g < (int)R::kGroups; ++g) {
                    const float s = qc::scale_value(rec[R::kKScales + tid * R::kGroups + g]);
                    float acc = 0.f;
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t word = *reinterpret_cast<const uint32_t *>(
                            rec + R::kKCodes + (g * kQPage + tid) * 16 + w * 4);
                        for (int e = 0; e < 8; ++e)
                            acc += s_q[g * 32 + w * 8 + e] *
                                   (float)((int)(word >> qc::code_shift(e) & 15u) - 8);
                    }
                    x += s * acc;
                }
                x *= a.scale;
            }
        } else if (tid < 64) {
            const int r = (t - pages) * 64 + tid;  // r steps above node i
            if (r < depth && (a.window <= 0 || r < a.window ||
                              ctx + (long long)depth - r - 1 < a.sinks)) {
                const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(a.k_tree) +
                                         (size_t)(off + s_path[r]) * a.kv_stride + kvh * D;
                x = 0.f;
                for (int c = 0; c < D; ++c) x += s_q[c] * __bfloat162float(k[c]);
                x *= a.scale;
            }
        }
        const float top = block_max(x, s_red);
        const float mn = fmaxf(m, top), ref = mn == ninf ? 0.f : mn;
        const float f = m == ninf ? 0.f : expf(m - ref);
        if (tid < 64) s_p[tid] = x == ninf ? 0.f : expf(x - ref);
        __syncthreads();
        m = mn;
        l *= f;
        o *= f;
        for (int j = 0; j < 64; ++j) {
            const float p = s_p[j];
            l += p;
            if (p == 0.f || tid >= D) continue;
            if (t < pages) {
                const uint32_t word = *reinterpret_cast<const uint32_t *>(
                    rec + R::kVCodes + ((j / 32) * D + tid) * 16 + ((j % 32) / 8) * 4);
                o += p * qc::scale_value(rec[R::kVScales + (tid / 32) * kQPage + j]) *
                     (float)((int)(word >> qc::code_shift(j & 7) & 15u) - 8);
            } else {
                const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v_tree) +
                                         (size_t)(off + s_path[(t - pages) * 64 + j]) *
                                             a.kv_stride + kvh * D;
                o += p * __bfloat162float(v[tid]);
            }
        }
        __syncthreads();
    }
    if (tid < D) {
        if (a.out_f32)
            of[tid] = o / l;
        else
            oh[tid] = __float2bfloat16_rn(o / l);
    }
}

}  // namespace

size_t qcache_attention_workspace_bytes(const QAttnArgs &a) {
    (void)a;
    return 0;
}

cudaError_t launch_qcache_attention(const QAttnArgs &a, cudaStream_t s) {
    const dim3 grid(a.B * a.max_nodes, a.H);
    return a.d == 64 ? launch_pdl(qcache_attention_kernel<64>, grid, dim3(128), 0, s, a)
                     : launch_pdl(qcache_attention_kernel<128>, grid, dim3(128), 0, s, a);
}

}  // namespace tv
