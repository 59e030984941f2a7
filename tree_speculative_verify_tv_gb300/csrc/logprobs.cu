// logprobs.cu -- log probabilities of given tokens, entropy and the most likely tokens.
//
//   m = max x, z = sum 2^{c (x - m)}, t = sum 2^{c (x - m)} c (x - m),   c = scale log2 e
//   logprob = scale (x_t - m) - ln z,   entropy = ln z - ln 2 t / z
// (LLM Primer VI ch. 9 §9.1: the distributions that accepted and emitted tokens are drawn from.)
//
// One pass: a thread keeps the maximum of what it has seen and z and t relative to it.  HBM
// bounds it: an element costs a 16th of a 16-byte load's issue, one exponential and about five
// other instructions.  A row is a CTA's, or, where rows are fewer than the SMs have room for, a
// cluster's, each CTA with a part of the row; partial results meet in distributed shared memory.
//
// Top tokens without another pass: threads form 64 groups with a maximum each.  The K-th largest
// of these, tau, is no larger than the K-th largest element, so the K are among the elements
// >= tau, which only the threads whose own maximum reaches tau have: those few read the turn of
// their maximum again, or all of their part if another turn reaches tau too (4096 rows of 131072
// bf16: 14 % more bytes from memory with whole parts, rows being far out of L2 by then).  Equal
// values at tau beyond what the list holds (constant or masked rows) are found in index order
// instead, and rows with a NaN, or a list that still overflows, by K searches.  Keys are (value,
// -index), so all of it is exact.  Where the finite values are in fewer than K groups tau is -inf and
// the list overflows: three times the time (256 rows of 131072 bf16, 8 alternatives, ten values each:
// 80 us; 31 with a hundred or all).
//
// Measured: those 4096 rows with 8 alternatives 178 us, 6.0 TB/s; 256 rows of 32000 bf16 9.7 us (2.4
// at the copy bandwidth) and one row of 50001 fp32 7.8 us, both of them latency
// (the first has 1.7 CTAs an SM, four rounds of loads each).
#include <cooperative_groups.h>

#include <type_traits>

#include "tv_internal.cuh"

namespace tv {
namespace {

namespace cg = cooperative_groups;

constexpr int kGroups = 64;
constexpr int kList = 1024;  // candidates that a CTA has room for
constexpr int kMaxTop = TV_LOGPROBS_MAX_TOP;
constexpr int kMaxCluster = 8;
constexpr int kUnroll = 4;   // 16-byte loads of a thread in flight
// Threads per SM that registers are kept to.  4096 rows of 131072 bf16, before a thread read
// one turn again: 193 us, with 1536 (spills) 208, with 1024 200.
constexpr int kPerSmThreads = 1280;

using Key = unsigned long long;

// Order of logits: larger value, larger key; a NaN above +inf (0xff800000), -0 equal to +0.  No
// key is all ones, a NaN at index 0 neither: that stands for "above every key".
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xfffffffeu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ Key make_key(float x, int i) {
    return ((Key)order_key(x) << 32) | (0xffffffffu - (uint32_t)i);
}
__device__ __forceinline__ int key_index(Key k) { return (int)(0xffffffffu - (uint32_t)k); }
__device__ __forceinline__ float key_value(Key k) {  // (a NaN's key gives some NaN)
    const uint32_t u = (uint32_t)(k >> 32);
    return __uint_as_float((u >> 31) ? u & 0x7fffffffu : ~u);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Elements of a 16-byte piece.
template <typename E>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
    static constexpr int kN = 8;
    static constexpr uint32_t kNothing = 0xFF80FF80u;  // -inf
    __device__ static float at(const uint4 &w, int e) {
        const uint32_t x = (&w.x)[e / 2];
        return __uint_as_float(e % 2 ? x & 0xFFFF0000u : x << 16);
    }
    __device__ static float largest(const uint4 (&w)[kUnroll]) {
        const auto b = [](uint32_t x) { return *reinterpret_cast<__nv_bfloat162 *>(&x); };
        __nv_bfloat162 m = b(kNothing);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            m = __hmax2(m, __hmax2(__hmax2(b(w[u].x), b(w[u].y)), __hmax2(b(w[u].z), b(w[u].w))));
        return fmaxf(__low2float(m), __high2float(m));
    }
};
template <>
struct Piece<float> {
    static constexpr int kN = 4;
    static constexpr uint32_t kNothing = 0xFF800000u;
    __device__ static float at(const uint4 &w, int e) { return __uint_as_float((&w.x)[e]); }
    __device__ static float largest(const uint4 (&w)[kUnroll]) {
        float m = -INFINITY;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) m = fmaxf(m, at(w[u], e));
        return m;
    }
};

// A maximum, and sums relative to it.
struct Sums {
    float m, z, t;
    // relative to `to` >= m instead
    __device__ void move(float to, float c) {
        if (m > -INFINITY && to != m) {
            const float d = (m - to) * c, f = ex2(d);
            t = f > 0.f ? f * fmaf(d, z, t) : 0.f * z;  // (z NaN stays)
            z *= f;
        }
        m = to;
    }
    __device__ void add(float x, float c) {
        if (x > m) move(x, c);
        const float y = (x - (m > -INFINITY ? m : 0.f)) * c, e = ex2(y);
        z += e;
        t = fmaf(e, fmaxf(y, -1.0e4f), t);
    }
};

// The sums of n parts, in order.
__device__ __forceinline__ Sums join(const Sums *parts, int n, float c) {
    Sums all{parts[0].m, 0.f, 0.f};
#pragma unroll 8
    for (int i = 1; i < n; ++i) all.m = fmaxf(all.m, parts[i].m);
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
        Sums p = parts[i];
        p.move(all.m, c);
        all.z += p.z;
        all.t += p.t;
    }
    return all;
}

template <int NT>
struct Shared {
    Sums sums[NT / 32];
    float group[kGroups];
    float tau;
    int count;
    Key best[NT / 32 + 1];
    Key list[kList + NT / 32 * kMaxTop];
    // read by the cluster's first CTA, and where it puts what it reads
    Sums total;
    Key top[kMaxTop];
    Sums totals[kMaxCluster];
    Key all[kMaxCluster * kMaxTop];
};

template <int NT>
__device__ __forceinline__ Key block_max(Key k, Key *s) {
    for (int o = 16; o > 0; o >>= 1) {
        const Key x = __shfl_xor_sync(0xffffffffu, k, o);
        k = x > k ? x : k;
    }
    if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = k;
    __syncthreads();
    for (int i = 0; i < NT / 32; ++i) k = s[i] > k ? s[i] : k;
    __syncthreads();
    return k;
}

// The K largest of `n` keys (all different) in falling order.
template <int NT>
__device__ __forceinline__ void rank_keys(const Key *list, int n, int K, Key *top) {
    for (int i = threadIdx.x; i < n; i += NT) {
        const Key k = list[i];
        int above = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) above += list[j] > k;
        if (above < K) top[above] = k;
    }
}

template <typename E, int NT>
__global__ void __launch_bounds__(NT, kPerSmThreads / NT) logprobs_kernel(LogprobsArgs a, int parts) {
    using P = Piece<E>;
    __shared__ Shared<NT> s;
    const int r = blockIdx.x / parts, part = blockIdx.x % parts;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    pdl_wait();
    pdl_launch_next();
    const int row = a.rows ? a.rows[r] : r;
    const int token = a.tokens ? a.tokens[r] : -1;
    if (tid == 0 && part == 0 && (row >= a.N || token >= a.V)) report(a.status, TV_ERR_SHAPE);
    if (row < 0 || row >= a.N) {  // (the same in every CTA of a cluster)
        if (part == 0) {
            if (tid == 0) {
                if (a.logprob) a.logprob[r] = 0.f;
                if (a.entropy) a.entropy[r] = 0.f;
            }
            for (int i = tid; i < a.top; i += NT) {
                a.top_token[(size_t)r * a.top + i] = -1;
                a.top_logprob[(size_t)r * a.top + i] = 0.f;
            }
        }
        return;
    }
    const E *x = static_cast<const E *>(a.logits) + (size_t)row * a.stride;
    const int V = a.V, K = min(a.top, V);
    const float c = fminf(a.scale * 1.44269504f, 3.0e38f);
    // elements ahead of the first 16-byte boundary, pieces, elements behind the last
    const int off = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(E));
    const int ahead = min((P::kN - off) % P::kN, V), pieces = (V - ahead) / P::kN;
    const int behind = V - ahead - pieces * P::kN;
    const uint4 *x4 = reinterpret_cast<const uint4 *>(x + ahead);
    const int per = (pieces + parts - 1) / parts;
    const int v0 = min(part * per, pieces), v1 = min(v0 + per, pieces);
    // this CTA's loose elements: a thread each
    const int loose = part == 0 && tid < ahead                 ? tid
                      : part == 0 && tid < ahead + behind      ? V - behind + (tid - ahead)
                                                               : -1;

    float at_token = 0.f;  // (on its way while the row is read)
    if (tid == 0 && part == 0 && token >= 0 && token < V) at_token = to_f32(x[token]);
    Sums mine{-INFINITY, 0.f, 0.f};
    // of this thread's turns: the largest value, where it came first, and the largest of the others
    float first = -INFINITY, second = -INFINITY;
    int where = v0 + tid;
    for (int v = v0 + tid; v < v1; v += NT * kUnroll) {
        uint4 w[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            w[u] = v + u * NT < v1 ? __ldg(x4 + v + u * NT)
                                   : make_uint4(P::kNothing, P::kNothing, P::kNothing, P::kNothing);
        const float most = P::largest(w);
        second = fmaxf(second, fminf(most, first));
        if (most > first) {
            first = most;
            where = v;
            mine.move(most, c);
        }
        const float m = mine.m > -INFINITY ? mine.m : 0.f;
        const Two less = two(-m, -m), c2 = two(c, c);
        Two z = 0, t = 0;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int e = 0; e < P::kN; e += 2) {
                const Two x2 = two(P::at(w[u], e), P::at(w[u], e + 1));
                const float2 y = halves(mul2(add2(x2, less), c2));
                const Two f = two(ex2(y.x), ex2(y.y));
                z = add2(z, f);
                // (-inf would meet its own exponential, 0)
                t = fma2(f, two(fmaxf(y.x, -1.0e4f), fmaxf(y.y, -1.0e4f)), t);
            }
        const float2 zs = halves(z), ts = halves(t);
        mine.z += zs.x + zs.y;
        mine.t += ts.x + ts.y;
    }
    if (loose >= 0) mine.add(to_f32(x[loose]), c);

    float g = mine.m;
    if (NT == 4 * kGroups) {
        g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 1));
        g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
        if (tid % 4 == 0) s.group[tid / 4] = g;
    } else {
        s.group[tid] = g;
    }
    float most = mine.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    mine.move(most, c);
    mine.z = warp_sum(mine.z);
    mine.t = warp_sum(mine.t);
    if (lane == 0) s.sums[warp] = mine;
    if (tid == 0) s.count = 0;
    __syncthreads();
    Sums sum = join(s.sums, NT / 32, c);
    const int mineN = (v1 - v0) * P::kN + (part == 0 ? ahead + behind : 0);  // elements here

    if (K > 0) {
        const int want = min(K, mineN);  // keys that this CTA has to give
        if (tid < K) s.top[tid] = 0;
        if (tid < kGroups) {
            const float v = s.group[tid];
            int above = 0;
#pragma unroll 16
            for (int j = 0; j < kGroups; ++j) {
                const float o = s.group[j];
                above += o > v || (o == v && j < tid);
            }
            if (above == K - 1) s.tau = v;
        }
        __syncthreads();
        const float tau = s.tau;
        bool search = sum.z != sum.z;  // a NaN or an infinity
        // Elements >= tau (or, if they are too many, > tau) into the list.
        const auto collect = [&](bool equal) {
            const auto put = [&](float y, int i) {
                if (equal ? y >= tau : y > tau) {
                    const int at = atomicAdd(&s.count, 1);
                    if (at < kList) s.list[at] = make_key(y, i);
                }
            };
            const bool has = equal ? first >= tau : first > tau;
            const bool more = equal ? second >= tau : second > tau;
            // a thread whose values all came in one turn reads that one again; the others' parts are
            // read by whole warps
            if (has && !more) {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int v = where + u * NT;
                    if (v < v1) {
                        const uint4 w = __ldg(x4 + v);
#pragma unroll
                        for (int e = 0; e < P::kN; ++e) put(P::at(w, e), ahead + v * P::kN + e);
                    }
                }
            }
            uint32_t who = __ballot_sync(0xffffffffu, more);
            while (who) {
                const int t = warp * 32 + __ffs(who) - 1;  // this thread's pieces
                who &= who - 1;
                for (int v = v0 + t + lane * NT; v < v1; v += 32 * NT) {
                    const uint4 w = __ldg(x4 + v);
#pragma unroll
                    for (int e = 0; e < P::kN; ++e) put(P::at(w, e), ahead + v * P::kN + e);
                }
            }
            if (loose >= 0) put(to_f32(x[loose]), loose);
            __syncthreads();
        };
        int n = 0;
        if (!search) {
            collect(true);
            n = s.count;
            if (n > kList) {
                __syncthreads();
                if (tid == 0) s.count = 0;
                __syncthreads();
                collect(false);
                n = s.count;
                __syncthreads();  // (read by all before it counts on)
                search = n > kList;
                if (!search && n < want) {
                    // the first few elements equal to tau, each warp in a stretch of its own
                    // (unsigned: a step may pass 2^31)
                    const uint32_t lo = part == 0 ? 0 : ahead + v0 * P::kN;
                    const uint32_t hi = part == parts - 1 ? V - (parts > 1 ? behind : 0)
                                                          : ahead + v1 * P::kN;
                    const uint32_t each = (hi - lo + NT / 32 - 1) / (NT / 32);
                    const uint32_t from = lo + warp * each, to = min(from + each, hi);
                    int found = 0;
                    for (uint32_t i = from; i < to && found < want; i += 32) {
                        const bool hit = i + lane < to && to_f32(x[i + lane]) == tau;
                        const uint32_t hits = __ballot_sync(0xffffffffu, hit);
                        const int at = found + __popc(hits & ((1u << lane) - 1));
                        if (hit && at < want) s.list[atomicAdd(&s.count, 1)] = make_key(tau, i + lane);
                        found += __popc(hits);
                    }
                    if (loose >= V - behind && parts > 1 && to_f32(x[loose]) == tau)
                        s.list[atomicAdd(&s.count, 1)] = make_key(tau, loose);
                    __syncthreads();
                    n = s.count;
                }
            }
        }
        if (!search) {
            rank_keys<NT>(s.list, n, K, s.top);
        } else {
            Key last = ~0ull;
            for (int j = 0; j < want; ++j) {
                Key best = 0;
                const auto look = [&](float y, int i) {
                    const Key k = make_key(y, i);
                    if (k < last && k > best) best = k;
                };
                for (int v = v0 + tid; v < v1; v += NT) {
                    const uint4 w = __ldg(x4 + v);
#pragma unroll
                    for (int e = 0; e < P::kN; ++e) look(P::at(w, e), ahead + v * P::kN + e);
                }
                if (loose >= 0) look(to_f32(x[loose]), loose);
                last = block_max<NT>(best, s.best);
                if (tid == 0) s.top[j] = last;
            }
        }
        __syncthreads();
    }

    const Key *top = s.top;
    if (parts > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        if (tid == 0) s.total = sum;
        cluster.sync();
        if (part == 0) {
            if (tid < parts) s.totals[tid] = *cluster.map_shared_rank(&s.total, tid);
            for (int i = tid; i < parts * K; i += NT)
                s.all[i] = cluster.map_shared_rank(s.top, i / K)[i % K];
        }
        cluster.sync();  // the others' shared memory has been read
        if (part != 0) return;
        // (parts with fewer elements than K have zeros, below every key and alike)
        for (int i = tid; i < parts * K; i += NT) {
            const Key k = s.all[i];
            int above = 0;
#pragma unroll 8
            for (int j = 0; j < parts * K; ++j) above += s.all[j] > k;
            if (k && above < K) s.list[above] = k;
        }
        __syncthreads();
        top = s.list;
        sum = join(s.totals, parts, c);
    }
    const float lnz = logf(sum.z), nan = __int_as_float(0x7fffffff);
    const bool bad = sum.z != sum.z, none = !bad && sum.m == -INFINITY;
    const auto logprob = [&](float v) {
        return bad ? nan : none ? -INFINITY : (v - sum.m) * a.scale - lnz;
    };
    if (tid == 0) {
        if (a.logprob)
            a.logprob[r] = token >= 0 && token < V ? logprob(at_token) : 0.f;
        if (a.entropy)
            a.entropy[r] = bad ? nan : none ? 0.f : lnz - 0.693147180559945309f * sum.t / sum.z;
    }
    for (int i = tid; i < K; i += NT) {
        a.top_token[(size_t)r * a.top + i] = key_index(top[i]);
        a.top_logprob[(size_t)r * a.top + i] = logprob(key_value(top[i]));
    }
}

template <typename E, int NT>
cudaError_t launch(const LogprobsArgs &a, int parts, cudaStream_t s) {
    if (parts == 1)
        return launch_pdl(logprobs_kernel<E, NT>, dim3((unsigned)a.R), dim3(NT), 0, s, a, 1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.R * parts));
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)parts;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, logprobs_kernel<E, NT>, a, parts);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Rows are cut until their CTAs would be more than kCut per SM, or parts shorter than kLeast bytes.
// 256 rows of 64 KB: 8.5 us uncut, 13.4 in halves (clusters start later, and meet twice).
constexpr int kCut = 2, kLeast = 8192;

template <typename E>
cudaError_t launch(const LogprobsArgs &a, cudaStream_t s) {
    const long long bytes = (long long)a.V * sizeof(E), sms = device_sms();
    int parts = 1;
    while (parts < kMaxCluster && (long long)a.R * parts * 2 <= kCut * sms && bytes / (parts * 2) >= kLeast)
        parts *= 2;
    // (rows of up to 4 KB leave most of 256 threads idle)
    return bytes <= 4096 ? launch<E, 64>(a, parts, s) : launch<E, 256>(a, parts, s);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsArgs &a, cudaStream_t s) {
    return a.dtype == TV_BF16 ? launch<__nv_bfloat16>(a, s) : launch<float>(a, s);
}

}  // namespace tv
