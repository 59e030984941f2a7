// qcache.cu -- rows quantised into the paged 4-bit KV cache, the accepted path's rows
// among them, and positions read back.
//
// The attention layers' share of committing a step (Bole summary page, "Core
// techniques" §2, restores only the accepted path's state; the branches of an attention
// layer differ only in their own keys and values).
#include "qcache.cuh"

namespace tv {
namespace {

constexpr int kThreadsQ = 256;

// Row blocks: request b's rows are cut where its positions enter a new page.  Block ids
// are handed out by base(b) = row_offsets[b] / 64 + 2 b, which leaves every request at
// least as many as it has pages to touch, so no counts have to be summed first.
__device__ __forceinline__ int block_base(const int32_t *offs, int b) {
    return max(offs[b], 0) / kQPage + 2 * b;
}

// The request that block id `blk` belongs to.
__device__ __forceinline__ int find_request(const int32_t *offs, int B, int blk) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (block_base(offs, mid) <= blk)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

struct RowBlock {
    int b, row, cnt;  // request, first packed row, rows (0: nothing to do)
    int pos;          // position of the first row
    bool fits;        // the request's rows lie in [0, 64 * max_pages); else pos counts from 0
};

// Block `blk` of a batch of rows; `tell` in one thread per block reports malformed input.
__device__ __forceinline__ RowBlock row_block(const QRowsArgs &a, int blk, bool tell) {
    RowBlock r{};
    int o, n;
    if (tell && blk < a.B && !request_range(a.offsets, blk, a.T, 0x7fffffff, o, n))
        report(a.status, TV_ERR_TREE);
    r.b = find_request(a.offsets, a.B, blk);
    if (!request_range(a.offsets, r.b, a.T, 0x7fffffff, o, n)) return r;
    const long long start = a.start[r.b], room = (long long)a.max_pages * kQPage;
    r.fits = start >= 0 && start + n <= room;
    if (tell && n > 0 && !r.fits) report(a.status, TV_ERR_SHAPE);
    const long long first = r.fits ? start : 0, page = first / kQPage;
    const int i = blk - block_base(a.offsets, r.b);  // the i-th page that the request touches
    const long long lo = max(first, (page + i) * kQPage);
    const long long hi = min(first + n, (page + i + 1) * kQPage);
    r.cnt = (int)max(0LL, hi - lo);
    r.row = o + (int)(lo - first);
    r.pos = (int)min(lo, 0x7fffffffLL);
    return r;
}

// The record of (request b, position pos, head h), or null (reported) for a bad page.
template <int D>
__device__ __forceinline__ uint8_t *record(const int32_t *table, int max_pages, int num_pages,
                                           int Hkv, uint8_t *cache, int b, int pos, int h,
                                           int32_t *status) {
    const int page = table[(size_t)b * max_pages + pos / kQPage];
    if (page < 0 || page >= num_pages) {
        report(status, TV_ERR_SHAPE);
        return nullptr;
    }
    return cache + ((size_t)page * Hkv + h) * qc::Rec<D>::kBytes;
}

// Rows src(0..cnt-1) of one group (lane = channel) into places off, off + 1, .. of a
// record.  V's words hold eight positions: a word that keeps some of its old codes is
// read first (a page being written has one writer per word, this warp).
template <int D, typename Row>
__device__ __forceinline__ void put_rows(uint8_t *rec, int g, int lane, int off, int cnt,
                                         const __nv_bfloat16 *k, const __nv_bfloat16 *v,
                                         Row row) {
    using R = qc::Rec<D>;
    const int c = g * kQGroup + lane;
    uint32_t word = 0, mask = 0;
    for (int m = 0; m < cnt; ++m) {
        const size_t at = row(m) + c;
        const uint32_t xk = __bfloat16_as_ushort(k[at]), xv = __bfloat16_as_ushort(v[at]);
        const uint32_t bk = qc::scale_byte(__reduce_max_sync(0xffffffffu, xk & 0x7FFFu));
        const uint32_t bv = qc::scale_byte(__reduce_max_sync(0xffffffffu, xv & 0x7FFFu));
        const int p = off + m;
        uint32_t w = qc::code(xk, qc::scale_inverse(bk)) << qc::code_shift(lane & 7);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) w |= __shfl_xor_sync(0xffffffffu, w, o);
        if ((lane & 7) == 0)
            *reinterpret_cast<uint32_t *>(rec + R::kKCodes + (g * kQPage + p) * 16 + lane / 2) = w;
        if (lane == 0) {
            rec[R::kKScales + p * R::kGroups + g] = (uint8_t)bk;
            rec[R::kVScales + g * kQPage + p] = (uint8_t)bv;
        }
        const int sh = qc::code_shift(p & 7);
        word |= qc::code(xv, qc::scale_inverse(bv)) << sh;
        mask |= 15u << sh;
        if ((p & 7) == 7 || m == cnt - 1) {
            uint32_t *dst = reinterpret_cast<uint32_t *>(
                rec + R::kVCodes + ((p / 32) * D + c) * 16 + ((p % 32) / 8) * 4);
            if (mask != 0xffffffffu) word |= *dst & ~mask;
            *dst = word;
            word = mask = 0;
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreadsQ) qcache_write_kernel(const QRowsArgs a) {
    constexpr int G = D / kQGroup;
    const int lane = threadIdx.x % 32;
    const long long unit = (long long)blockIdx.x * (kThreadsQ / 32) + threadIdx.x / 32;
    const int g = (int)(unit % G), h = (int)(unit / G % a.Hkv);
    const long long blk = unit / G / a.Hkv;
    pdl_wait();
    pdl_launch_next();
    if (blk >= a.T / kQPage + 2LL * a.B) return;
    const RowBlock r = row_block(a, (int)blk, lane == 0 && g == 0 && h == 0);
    if (r.cnt == 0 || !r.fits) return;
    uint8_t *rec = record<D>(a.table, a.max_pages, a.num_pages, a.Hkv, a.cache, r.b, r.pos, h,
                             a.status);
    if (!rec) return;
    const size_t first = (size_t)r.row * a.stride + (size_t)h * D;
    put_rows<D>(rec, g, lane, r.pos % kQPage, r.cnt, static_cast<const __nv_bfloat16 *>(a.k),
                static_cast<const __nv_bfloat16 *>(a.v),
                [&](int m) { return first + (size_t)m * a.stride; });
}

template <int D>
__global__ void __launch_bounds__(kThreadsQ) qcache_read_kernel(const QRowsArgs a) {
    using R = qc::Rec<D>;
    constexpr int G = D / kQGroup;
    const int lane = threadIdx.x % 32;
    const long long unit = (long long)blockIdx.x * (kThreadsQ / 32) + threadIdx.x / 32;
    const int g = (int)(unit % G), h = (int)(unit / G % a.Hkv);
    const long long blk = unit / G / a.Hkv;
    pdl_wait();
    pdl_launch_next();
    if (blk >= a.T / kQPage + 2LL * a.B) return;
    const bool tell = lane == 0 && g == 0 && h == 0;
    const RowBlock r = row_block(a, (int)blk, tell);
    if (r.cnt == 0) return;
    const int len = a.len[r.b];
    const bool len_ok = len >= 0 && len <= (long long)a.max_pages * kQPage;
    if (tell && !len_ok) report(a.status, TV_ERR_SHAPE);
    const int live = r.fits && len_ok ? min(max(len - r.pos, 0), r.cnt) : 0;
    const uint8_t *rec = live > 0 ? record<D>(a.table, a.max_pages, a.num_pages, a.Hkv, a.cache,
                                              r.b, r.pos, h, a.status)
                                  : nullptr;
    const int c = g * kQGroup + lane, sh = qc::code_shift(lane & 7);
    __nv_bfloat16 *k = static_cast<__nv_bfloat16 *>(a.k), *v = static_cast<__nv_bfloat16 *>(a.v);
    for (int m = 0; m < r.cnt; ++m) {
        const size_t at = (size_t)(r.row + m) * a.stride + (size_t)h * D + c;
        float xk = 0.f, xv = 0.f;
        if (rec && m < live) {
            const int p = r.pos % kQPage + m;
            const uint32_t wk = *reinterpret_cast<const uint32_t *>(
                rec + R::kKCodes + (g * kQPage + p) * 16 + lane / 8 * 4);
            const uint32_t wv = *reinterpret_cast<const uint32_t *>(
                rec + R::kVCodes + ((p / 32) * D + c) * 16 + ((p % 32) / 8) * 4);
            xk = qc::scale_value(rec[R::kKScales + p * R::kGroups + g]) *
                 (float)((int)(wk >> sh & 15u) - 8);
            xv = qc::scale_value(rec[R::kVScales + g * kQPage + p]) *
                 (float)((int)(wv >> qc::code_shift(p & 7) & 15u) - 8);
        }
        k[at] = __float2bfloat16_rn(xk);  // exact: at most 7 significant bits
        v[at] = __float2bfloat16_rn(xv);
    }
}

// One CTA per request, so that the lengths may advance in place: everything that reads
// ctx_len has read it before the barrier.
template <int D>
__global__ void __launch_bounds__(kThreadsQ) qcache_commit_kernel(const QCommitArgs a) {
    constexpr int G = D / kQGroup;
    __shared__ int s_node[kMaxDepth];
    __shared__ int s_bad;
    const int b = blockIdx.x, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    pdl_wait();
    pdl_launch_next();
    int off, n;
    const bool range = request_range(a.node_offsets, b, a.T, a.max_nodes, off, n);
    const int L = a.accept_len[b], ctx = a.ctx_len[b];
    const long long room = (long long)a.max_pages * kQPage;
    const bool tree_ok = range && L >= 0 && L <= a.max_depth;
    const bool len_ok = ctx >= 0 && ctx + (long long)max(L, 0) <= room;
    if (threadIdx.x == 0) s_bad = !tree_ok ? TV_ERR_TREE : !len_ok ? TV_ERR_SHAPE : 0;
    __syncthreads();
    if (tree_ok && len_ok && (int)threadIdx.x < L) {
        const int m = threadIdx.x, node = a.path[(size_t)b * a.max_depth + m];
        s_node[m] = off + node;
        if (node < 0 || node >= n) s_bad = TV_ERR_TREE;
        const int page = a.table[(size_t)b * a.max_pages + (ctx + m) / kQPage];
        if (page < 0 || page >= a.num_pages) atomicCAS(&s_bad, 0, TV_ERR_SHAPE);
    }
    __syncthreads();
    const int bad = s_bad;
    if (threadIdx.x == 0) {
        a.new_len[b] = bad ? ctx : ctx + L;
        if (bad) report(a.status, bad);
    }
    if (bad) return;
    for (int u = warp; u < a.Hkv * G; u += kThreadsQ / 32) {
        const int g = u % G, h = u / G;
        for (int m0 = 0; m0 < L;) {  // the pages that the path touches: one or two
            const int pos = ctx + m0, cnt = min(L - m0, kQPage - pos % kQPage);
            const int page = a.table[(size_t)b * a.max_pages + pos / kQPage];
            uint8_t *rec = a.cache + ((size_t)page * a.Hkv + h) * qc::Rec<D>::kBytes;
            put_rows<D>(rec, g, lane, pos % kQPage, cnt, static_cast<const __nv_bfloat16 *>(a.k),
                        static_cast<const __nv_bfloat16 *>(a.v), [&](int m) {
                            return (size_t)s_node[m0 + m] * a.stride + (size_t)h * D;
                        });
            m0 += cnt;
        }
    }
}

template <typename Kern>
cudaError_t launch_rows(Kern kern, const QRowsArgs &a, cudaStream_t s) {
    const long long units = (a.T / kQPage + 2LL * a.B) * a.Hkv * (a.d / kQGroup);
    const unsigned grid = (unsigned)((units + kThreadsQ / 32 - 1) / (kThreadsQ / 32));
    return launch_pdl(kern, dim3(grid), dim3(kThreadsQ), 0, s, a);
}

}  // namespace

cudaError_t launch_qcache_write(const QRowsArgs &a, cudaStream_t s) {
    return a.d == 64 ? launch_rows(qcache_write_kernel<64>, a, s)
                     : launch_rows(qcache_write_kernel<128>, a, s);
}

cudaError_t launch_qcache_read(const QRowsArgs &a, cudaStream_t s) {
    return a.d == 64 ? launch_rows(qcache_read_kernel<64>, a, s)
                     : launch_rows(qcache_read_kernel<128>, a, s);
}

cudaError_t launch_qcache_commit(const QCommitArgs &a, cudaStream_t s) {
    return a.d == 64 ? launch_pdl(qcache_commit_kernel<64>, dim3(a.B), dim3(kThreadsQ), 0, s, a)
                     : launch_pdl(qcache_commit_kernel<128>, dim3(a.B), dim3(kThreadsQ), 0, s, a);
}

}  // namespace tv
