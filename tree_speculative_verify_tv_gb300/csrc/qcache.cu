// qcache.cu -- rows quantised into the paged 4-bit KV cache, the accepted path's rows
// among them, and positions read back.
//
// The attention layers' share of committing a step (Bole summary page, "Core
// techniques" §2, restores only the accepted path's state; the branches of an attention
// layer differ only in their own keys and values).
#include "qcache.cuh"

namespace tv {
namespace {

constexpr int kThreadsQ = 128;
constexpr int kWriteCtas = 8;  // writing CTAs per SM that registers leave room for

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

// What a lane holds of a row: 8 channels (one word of K's codes), D / 8 lanes to a row.
// Scale byte of the 32-channel group of four neighbouring lanes, from their pieces.
__device__ __forceinline__ uint32_t group_scale(const uint4 &x) {
    const uint32_t m = 0x7FFF7FFFu;
    uint32_t y = qc::max2(qc::max2(x.x & m, x.y & m), qc::max2(x.z & m, x.w & m));
    y = qc::max2(y, __shfl_xor_sync(0xffffffffu, y, 1));
    y = qc::max2(y, __shfl_xor_sync(0xffffffffu, y, 2));
    return qc::scale_byte(max(y & 0xFFFFu, y >> 16));
}

__device__ __forceinline__ float low_half(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float high_half(uint32_t x) {
    return __uint_as_float(x & 0xFFFF0000u);
}

// The piece with values beyond the range of the largest step clamped (a rare branch).
__device__ __forceinline__ uint4 in_range(uint4 x, uint32_t b) {
    if (__any_sync(0xffffffffu, b == 254)) {
        if (b == 254)
            x = make_uint4(qc::clamp_pair(x.x), qc::clamp_pair(x.y), qc::clamp_pair(x.z),
                           qc::clamp_pair(x.w));
    }
    return x;
}

// K rows from .. cnt - 1 of those that go to places off + row: a warp takes 32 / (D / 8)
// rows at a time, kBatch loads in flight per lane.
template <int D, typename Row>
__device__ __forceinline__ void put_k(uint8_t *rec, int lane, int off, int from, int cnt,
                                      const __nv_bfloat16 *k, Row row) {
    using R = qc::Rec<D>;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kBatch = 4;
    const int w = lane % kLanes, g = w / 4;
    for (int m0 = from + lane / kLanes; m0 < cnt + lane / kLanes; m0 += kRows * kBatch) {
        uint4 x[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int m = m0 + u * kRows;
            x[u] = make_uint4(0, 0, 0, 0);
            if (m < cnt) x[u] = *reinterpret_cast<const uint4 *>(k + row(m) + w * 8);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int m = m0 + u * kRows, p = off + m;
            const uint32_t b = group_scale(x[u]);
            const float inv = qc::scale_inverse(b);
            const uint4 y = in_range(x[u], b);
            const uint32_t h[4] = {y.x, y.y, y.z, y.w};
            uint32_t word = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                word = qc::put_code(word, low_half(h[e]), inv, qc::code_shift(2 * e));
                word = qc::put_code(word, high_half(h[e]), inv, qc::code_shift(2 * e + 1));
            }
            // the row's scale bytes in its first lane
            uint32_t sc = w % 4 == 0 ? b << (8 * g) : 0;
            sc |= __shfl_xor_sync(0xffffffffu, sc, 4);
            if (D == 128) sc |= __shfl_xor_sync(0xffffffffu, sc, 8);
            if (m < cnt) {
                *reinterpret_cast<uint32_t *>(rec + R::kKCodes + (g * kQPage + p) * 16 +
                                              w % 4 * 4) = word;
                if (w == 0) {
                    if (D == 128)
                        *reinterpret_cast<uint32_t *>(rec + R::kKScales + p * 4) = sc;
                    else
                        *reinterpret_cast<uint16_t *>(rec + R::kKScales + p * 2) = (uint16_t)sc;
                }
            }
        }
    }
}

// V rows [off, off + cnt) of a record, as far as they fall into part `part` of its places
// (half a page at D = 128, all of it at D = 64): a lane takes its 8 channels at 16
// consecutive positions, so that it ends with whole words, of 8 positions each.  Words that
// keep some of their old codes are read first (a word being written has one writer, this
// lane).
template <int D, typename Row>
__device__ __forceinline__ void put_v(uint8_t *rec, int lane, int part, int off, int cnt,
                                      const __nv_bfloat16 *v, Row row) {
    using R = qc::Rec<D>;
    constexpr int kLanes = D / 8, kPos = 16, kBatch = 8;
    const int o = lane % kLanes, p0 = part * kPos * (32 / kLanes) + lane / kLanes * kPos, g = o / 4;
    const int lo = max(off - p0, 0), hi = min(off + cnt - p0, kPos);  // of this lane's places
    uint32_t word[kPos / 8][8];
#pragma unroll
    for (int q = 0; q < kPos / 8; ++q) {
#pragma unroll
        for (int c = 0; c < 8; ++c) word[q][c] = 0;
        if (!__any_sync(0xffffffffu, 8 * q < hi && 8 * q + 8 > lo)) continue;
        uint4 x[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = 8 * q + u;
            x[u] = make_uint4(0, 0, 0, 0);
            if (i >= lo && i < hi)
                x[u] = *reinterpret_cast<const uint4 *>(v + row(p0 + i - off) + o * 8);
        }
        uint32_t bytes[2] = {0, 0};
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const uint32_t b = group_scale(x[u]);
            const float inv = qc::scale_inverse(b);
            const uint4 y = in_range(x[u], b);
            const uint32_t h[4] = {y.x, y.y, y.z, y.w};
            bytes[u / 4] |= b << (8 * (u % 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                word[q][2 * e] = qc::put_code(word[q][2 * e], low_half(h[e]), inv,
                                              qc::code_shift(u));
                word[q][2 * e + 1] = qc::put_code(word[q][2 * e + 1], high_half(h[e]), inv,
                                                  qc::code_shift(u));
            }
        }
        // the group's scale bytes, by its first lane
        if (o % 4 == 0) {
            uint8_t *sc = rec + R::kVScales + g * kQPage + p0 + 8 * q;
            if (lo <= 8 * q && hi >= 8 * q + 8) {
                *reinterpret_cast<uint2 *>(sc) = make_uint2(bytes[0], bytes[1]);
            } else {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (8 * q + u >= lo && 8 * q + u < hi)
                        sc[u] = (uint8_t)(bytes[u / 4] >> (8 * (u % 4)));
            }
        }
    }
    if (lo >= hi) return;
    // words of positions [8 q, 8 q + 8): which codes are new
    uint32_t mask[kPos / 8];
    bool all = true;
#pragma unroll
    for (int q = 0; q < kPos / 8; ++q) {
        mask[q] = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (8 * q + u >= lo && 8 * q + u < hi) mask[q] |= 15u << qc::code_shift(u);
        all = all && mask[q] == 0xffffffffu;
    }
    uint32_t *dst = reinterpret_cast<uint32_t *>(rec + R::kVCodes + ((p0 / 32) * D + 8 * o) * 16 +
                                                 p0 % 32 / 8 * 4);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        uint32_t *d = dst + 4 * c;
        if (!all) {
#pragma unroll
            for (int q = 0; q < kPos / 8; ++q)
                if (mask[q] != 0xffffffffu)
                    word[q][c] = (word[q][c] & mask[q]) | (d[q] & ~mask[q]);
        }
        *reinterpret_cast<uint2 *>(d) = make_uint2(word[0][c], word[1][c]);
    }
}

// One warp per part of K or V of a (block, head): half a page (of V at D = 64: all of it).
//
// 65536 rows of 8 heads x 128 channels: 81 us for the 268 MB read and the 71 MB written,
// 4.2 TB/s, 63 % of the copy bandwidth.  The arithmetic pipe is the busiest unit (63 %; some
// 20 of its operations per pair of values), with the loads' latency beside it: eight CTAs of
// four warps per SM need 64 registers, and seven without the one spilled value took 84 us.  A
// warp per whole page of K or V took 106 us, a thread per group of channels 330.
template <int D>
__global__ void __launch_bounds__(kThreadsQ, kWriteCtas) qcache_write_kernel(const QRowsArgs a) {
    constexpr int kParts = 2, kVParts = D / 64;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int h = blockIdx.x % a.Hkv, blk = blockIdx.x / a.Hkv;
    pdl_wait();
    pdl_launch_next();
    const RowBlock r = row_block(a, blk, threadIdx.x == 0 && h == 0);
    if (r.cnt == 0 || !r.fits) return;
    uint8_t *rec = record<D>(a.table, a.max_pages, a.num_pages, a.Hkv, a.cache, r.b, r.pos, h,
                             a.status);
    if (!rec) return;
    const size_t first = (size_t)r.row * a.stride + (size_t)h * D;
    auto row = [&](int m) { return first + (size_t)m * a.stride; };
    const int off = r.pos % kQPage;
    if (warp < kParts) {
        const int half = (r.cnt + kParts - 1) / kParts;
        put_k<D>(rec, lane, off, warp * half, min(r.cnt, (warp + 1) * half),
                 static_cast<const __nv_bfloat16 *>(a.k), row);
    } else if (warp < kParts + kVParts) {
        put_v<D>(rec, lane, warp - kParts, off, r.cnt, static_cast<const __nv_bfloat16 *>(a.v),
                 row);
    }
}

// One warp per K or V of a (block, head): a lane gives 8 channels of a row, 16 bytes.
// 65536 positions of 8 heads x 128 channels: 58.6 us for 71 MB in and 268 MB out, 5.8 TB/s,
// 87 % of the copy bandwidth, which bounds it.
template <int D>
__global__ void __launch_bounds__(kThreadsQ) qcache_read_kernel(const QRowsArgs a) {
    using R = qc::Rec<D>;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kPos = kQPage * kLanes / 32, kBatch = 8;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const long long unit = (long long)blockIdx.x * (kThreadsQ / 64) + warp / 2;
    const int h = (int)(unit % a.Hkv);
    const long long blk = unit / a.Hkv;
    pdl_wait();
    pdl_launch_next();
    if (blk >= a.T / kQPage + 2LL * a.B) return;
    const bool tell = lane == 0 && warp % 2 == 0 && h == 0;
    const RowBlock r = row_block(a, (int)blk, tell);
    if (r.cnt == 0) return;
    const int len = a.len[r.b];
    const bool len_ok = len >= 0 && len <= (long long)a.max_pages * kQPage;
    if (tell && !len_ok) report(a.status, TV_ERR_SHAPE);
    int live = r.fits && len_ok ? min(max(len - r.pos, 0), r.cnt) : 0;
    const uint8_t *rec = live > 0 ? record<D>(a.table, a.max_pages, a.num_pages, a.Hkv, a.cache,
                                              r.b, r.pos, h, a.status)
                                  : nullptr;
    if (!rec) live = 0;
    const int off = r.pos % kQPage, w = lane % kLanes, g = w / 4;
    const size_t first = (size_t)r.row * a.stride + (size_t)h * D + w * 8;
    if (warp % 2 == 0) {
        __nv_bfloat16 *k = static_cast<__nv_bfloat16 *>(a.k) + first;
        for (int m0 = lane / kLanes; m0 < r.cnt; m0 += kRows * kBatch) {
            uint32_t word[kBatch], b[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int m = m0 + u * kRows, p = off + m;
                word[u] = 0x88888888u;  // zeros
                b[u] = 0;
                if (m < live) {
                    word[u] = *reinterpret_cast<const uint32_t *>(
                        rec + R::kKCodes + (g * kQPage + p) * 16 + w % 4 * 4);
                    b[u] = rec[R::kKScales + p * R::kGroups + g];
                }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int m = m0 + u * kRows;
                const uint32_t s2 = qc::scale_pair(b[u]), ms = qc::minus_136(s2);
                if (m < r.cnt)
                    *reinterpret_cast<uint4 *>(k + (size_t)m * a.stride) = make_uint4(
                        qc::value_pair(word[u], 0, s2, ms), qc::value_pair(word[u], 1, s2, ms),
                        qc::value_pair(word[u], 2, s2, ms), qc::value_pair(word[u], 3, s2, ms));
            }
        }
        return;
    }
    // V: this lane's 8 channels at kPos positions, words of 8 positions per channel
    const int p0 = lane / kLanes * kPos;
    __nv_bfloat16 *v = static_cast<__nv_bfloat16 *>(a.v) + first;
    const int lo = max(off - p0, 0), hi = min(off + r.cnt - p0, kPos);
    const int end = min(off + live - p0, kPos);  // rows from here on are zeros
    if (lo >= hi) return;
    uint32_t word[8][kPos / 8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const uint8_t *src = rec + R::kVCodes + ((p0 / 32) * D + 8 * w + c) * 16 + p0 % 32 / 8 * 4;
#pragma unroll
        for (int q = 0; q < kPos / 8; ++q) word[c][q] = 0x88888888u;
        if (end > lo) {
            if constexpr (kPos == 32) {
                const uint4 x = *reinterpret_cast<const uint4 *>(src);
                word[c][0] = x.x;
                word[c][1] = x.y;
                word[c][2] = x.z;
                word[c][3] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(src);
                word[c][0] = x.x;
                word[c][1] = x.y;
            }
        }
    }
#pragma unroll
    for (int q = 0; q < kPos / 8; ++q) {
        if (8 * q >= hi || 8 * q + 8 <= lo) continue;
        uint32_t bytes[2] = {0, 0};
        if (end > lo) {
            const uint2 x = *reinterpret_cast<const uint2 *>(rec + R::kVScales + g * kQPage + p0 + 8 * q);
            bytes[0] = x.x;
            bytes[1] = x.y;
        }
        // even positions have their nibbles in the words' low halves, odd ones in the high
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {
            uint32_t pair[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                pair[e] = __byte_perm(word[2 * e][q], word[2 * e + 1][q], odd ? 0x7632 : 0x5410);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int u = 2 * p + odd, i = 8 * q + u;
                const uint32_t b = (bytes[u / 4] >> (8 * (u % 4))) & 0xFFu;
                const uint32_t s2 = qc::scale_pair(b), ms = qc::minus_136(s2);
                uint4 y = make_uint4(qc::value_pair(pair[0], p, s2, ms),
                                     qc::value_pair(pair[1], p, s2, ms),
                                     qc::value_pair(pair[2], p, s2, ms),
                                     qc::value_pair(pair[3], p, s2, ms));
                if (i >= end) y = make_uint4(0, 0, 0, 0);
                if (i >= lo && i < hi)
                    *reinterpret_cast<uint4 *>(v + (size_t)(p0 + i - off) * a.stride) = y;
            }
        }
    }
}

// One CTA per request, so that the lengths may advance in place; latency bounds it (three
// dependent loads, then the rows): with the positions read back 13.7 us for 16 requests, 47
// for 128 requests of 64-node trees.  Everything that reads
// ctx_len has read it before the barrier.  A warp per K, or part of V, of a head: 24 of them
// at 8 heads of 128 channels (16 warps, and two rounds, took 1.6 us longer per call).
constexpr int kThreadsCommit = 768;

template <int D>
__global__ void __launch_bounds__(kThreadsCommit) qcache_commit_kernel(const QCommitArgs a) {
    __shared__ int s_node[kMaxDepth], s_page[2];
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
        s_page[(ctx + m) / kQPage - ctx / kQPage] = page;
    }
    __syncthreads();
    const int bad = s_bad;
    if (threadIdx.x == 0) {
        a.new_len[b] = bad ? ctx : ctx + L;
        if (bad) report(a.status, bad);
    }
    if (bad) return;
    constexpr int kTasks = 1 + D / 64;  // K, and the parts of V
    for (int u = warp; u < a.Hkv * kTasks; u += kThreadsCommit / 32) {
        const int h = u / kTasks, part = u % kTasks - 1;
        for (int m0 = 0; m0 < L;) {  // the pages that the path touches: one or two
            const int pos = ctx + m0, cnt = min(L - m0, kQPage - pos % kQPage);
            uint8_t *rec = a.cache +
                           ((size_t)s_page[pos / kQPage - ctx / kQPage] * a.Hkv + h) *
                               qc::Rec<D>::kBytes;
            auto row = [&](int m) { return (size_t)s_node[m0 + m] * a.stride + (size_t)h * D; };
            if (part < 0)
                put_k<D>(rec, lane, pos % kQPage, 0, cnt, static_cast<const __nv_bfloat16 *>(a.k),
                         row);
            else
                put_v<D>(rec, lane, part, pos % kQPage, cnt,
                         static_cast<const __nv_bfloat16 *>(a.v), row);
            m0 += cnt;
        }
    }
}

}  // namespace

cudaError_t launch_qcache_write(const QRowsArgs &a, cudaStream_t s) {
    const dim3 grid((unsigned)((a.T / kQPage + 2LL * a.B) * a.Hkv));
    return a.d == 64 ? launch_pdl(qcache_write_kernel<64>, grid, dim3(kThreadsQ), 0, s, a)
                     : launch_pdl(qcache_write_kernel<128>, grid, dim3(kThreadsQ), 0, s, a);
}

cudaError_t launch_qcache_read(const QRowsArgs &a, cudaStream_t s) {
    const long long units = (a.T / kQPage + 2LL * a.B) * a.Hkv;
    const dim3 grid((unsigned)((units + kThreadsQ / 64 - 1) / (kThreadsQ / 64)));
    return a.d == 64 ? launch_pdl(qcache_read_kernel<64>, grid, dim3(kThreadsQ), 0, s, a)
                     : launch_pdl(qcache_read_kernel<128>, grid, dim3(kThreadsQ), 0, s, a);
}

cudaError_t launch_qcache_commit(const QCommitArgs &a, cudaStream_t s) {
    return a.d == 64
               ? launch_pdl(qcache_commit_kernel<64>, dim3(a.B), dim3(kThreadsCommit), 0, s, a)
               : launch_pdl(qcache_commit_kernel<128>, dim3(a.B), dim3(kThreadsCommit), 0, s, a);
}

}  // namespace tv
