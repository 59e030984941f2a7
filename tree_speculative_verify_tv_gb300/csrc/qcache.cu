// qcache.cu -- rows quantised into the paged 4-bit KV cache, the accepted path's rows
// among them, and positions read back.
//
// The attention layers' share of committing a step (Bole summary page, "Core
// techniques" §2, restores only the accepted path's state; the branches of an attention
// layer differ only in their own keys and values).
#include "qcache.cuh"
#include "tc_ptx.cuh"

namespace tv {
namespace {

constexpr int kThreadsQ = 128;
constexpr int kWriteCtas = 8;  // writing CTAs per SM that registers leave room for
constexpr int kStage = 8;      // pieces of a lane in flight

// Row blocks: request b's rows are cut where its positions enter a new page.  Block ids
// are handed out by base(b) = row_offsets[b] / 64 + 2 b, which leaves every request at
// least as many as it has pages to touch, so no counts have to be summed first.
__device__ __forceinline__ int block_base(const int32_t *offs, int b) {
    return max(offs[b], 0) / kQPage + 2 * b;
}

// The request that block id `blk` belongs to, by a whole warp: each round of loads leaves a
// 32nd of the requests (a binary search is a chain of five loads for 32 of them).
__device__ __forceinline__ int find_request(const int32_t *offs, int B, int blk) {
    const int lane = threadIdx.x % 32;
    int lo = 0, n = B;
    while (n > 1) {
        const int step = (n + 31) / 32, at = lane * step;
        const uint32_t begun =
            __ballot_sync(0xffffffffu, at < n && block_base(offs, lo + at) <= blk);
        const int k = max(__popc(begun) - 1, 0) * step;
        lo += k;
        n = min(step, n - k);
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

// The piece with values beyond the range of the largest step clamped, and zeros for that of a
// group with a NaN (a rare branch; the others' values are within the range anyway).
__device__ __forceinline__ uint4 in_range(uint4 x, uint32_t b) {
    if (__any_sync(0xffffffffu, b >= 254)) {
        const uint32_t keep = b == 255 ? 0u : 0xffffffffu;
        x = make_uint4(qc::clamp_pair(x.x) & keep, qc::clamp_pair(x.y) & keep,
                       qc::clamp_pair(x.z) & keep, qc::clamp_pair(x.w) & keep);
    }
    return x;
}

// A lane's pieces on their way to the codes: asynchronous copies into shared memory of its
// own, so that kStage loads are in flight from a short loop.  (Loads into registers needed
// the loops around them unrolled: 52 KB of code, more than the instruction cache holds, and
// 2 us more on a call of ragged chunks, 4 on 65536 rows.)
struct Staged {
    uint4 *at;  // the warp's [kStage][32]
    int lane;
    __device__ void load(int i, const __nv_bfloat16 *from) const {
        ptx::cp_async_16(ptx::smem_addr(at + i * 32 + lane), from);
    }
    __device__ uint4 operator[](int i) const { return at[i * 32 + lane]; }
};

// K rows from .. cnt - 1 of those that go to places off + row: a warp takes 32 / (D / 8)
// rows at a time.
template <int D, typename Row>
__device__ __forceinline__ void put_k(uint8_t *rec, const Staged &stage, int off, int from,
                                      int cnt, const __nv_bfloat16 *k, Row row) {
    using R = qc::Rec<D>;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    const int lane = stage.lane, w = lane % kLanes, g = w / 4;
#pragma unroll 1
    for (int m0 = from; m0 < cnt; m0 += kRows * kStage) {
        const int n = min(kStage, (cnt - m0 + kRows - 1) / kRows), first = m0 + lane / kLanes;
#pragma unroll 2
        for (int i = 0; i < n; ++i) {
            const int m = first + i * kRows;
            if (m < cnt) stage.load(i, k + row(m) + w * 8);
        }
        ptx::cp_async_wait_all();
        uint8_t *codes = rec + R::kKCodes + (g * kQPage + off + first) * 16 + w % 4 * 4;
        uint8_t *scales = rec + R::kKScales + (off + first) * R::kGroups;
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const uint4 x = stage[i];
            const uint32_t b = group_scale(x);
            const float inv = qc::scale_inverse(b);
            const uint4 y = in_range(x, b);
            const uint32_t h[4] = {y.x, y.y, y.z, y.w};
            uint32_t word = qc::kNoCodes;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                word = qc::put_code(word, low_half(h[e]), inv, 1u << qc::code_shift(2 * e));
                word = qc::put_code(word, high_half(h[e]), inv, 1u << qc::code_shift(2 * e + 1));
            }
            // the row's scale bytes in its first lane
            uint32_t sc = w % 4 == 0 ? b << (8 * g) : 0;
            sc |= __shfl_xor_sync(0xffffffffu, sc, 4);
            if (D == 128) sc |= __shfl_xor_sync(0xffffffffu, sc, 8);
            if (first + i * kRows < cnt) {
                *reinterpret_cast<uint32_t *>(codes + i * kRows * 16) = word;
                if (w == 0) {
                    if (D == 128)
                        *reinterpret_cast<uint32_t *>(scales + i * kRows * 4) = sc;
                    else
                        *reinterpret_cast<uint16_t *>(scales + i * kRows * 2) = (uint16_t)sc;
                }
            }
        }
    }
}

// The bits of elements [from, to) of a word of eight codes.
__device__ __forceinline__ uint32_t code_mask(int from, int to) {
    from = min(max(from, 0), 8), to = min(max(to, from), 8);
    const uint32_t e = (1u << to) - (1u << from);  // a bit per element, then spread
    const uint32_t s = (e & 3u) | (e & 12u) << 2 | (e & 48u) << 4 | (e & 192u) << 6;
    return (s & 0x1111u) * 15u | ((s >> 1) & 0x1111u) * 0xF0000u;
}

// V rows [off, off + cnt) of a record, as far as they fall into part `part` of its places
// (half a page at D = 128, all of it at D = 64): a lane takes its 8 channels at 16
// consecutive positions, so that it ends with whole words, of 8 positions each.  Words that
// keep some of their old codes are read first (a word being written has one writer, this
// lane).
template <int D, typename Row>
__device__ __forceinline__ void put_v(uint8_t *rec, const Staged &stage, int part, int off,
                                      int cnt, const __nv_bfloat16 *v, Row row) {
    using R = qc::Rec<D>;
    constexpr int kLanes = D / 8, kPos = 16;
    static_assert(kStage == 8, "a word of positions");
    const int lane = stage.lane, o = lane % kLanes, g = o / 4;
    const int p0 = part * kPos * (32 / kLanes) + lane / kLanes * kPos;
    const int lo = max(off - p0, 0), hi = min(off + cnt - p0, kPos);  // of this lane's places
    if (!__any_sync(0xffffffffu, lo < hi)) return;
    uint32_t first[8], word[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) word[c] = 0;
#pragma unroll 1
    for (int q = 0; q < kPos / 8; ++q) {
#pragma unroll 2
        for (int i = 0; i < kStage; ++i) {
            const int p = 8 * q + i;
            if (p >= lo && p < hi) stage.load(i, v + row(p0 + p - off) + o * 8);
        }
        ptx::cp_async_wait_all();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            first[c] = word[c];
            word[c] = qc::kNoCodes;
        }
        if (!__any_sync(0xffffffffu, 8 * q < hi && 8 * q + 8 > lo)) continue;
        uint32_t bytes[2] = {0, 0};  // eight scale bytes, moved down by two at a time
#pragma unroll
        for (int u = 0; u < 8; u += 2) {
            uint32_t two[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                // (a place without a row has whatever is staged: it is not stored)
                const uint4 x = stage[u + s];
                const uint32_t b = two[s] = group_scale(x);
                const float inv = qc::scale_inverse(b);
                const uint4 y = in_range(x, b);
                const uint32_t h[4] = {y.x, y.y, y.z, y.w};
                const uint32_t place = 1u << (2 * u + 16 * s);  // code_shift(u + s)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    word[2 * e] = qc::put_code(word[2 * e], low_half(h[e]), inv, place);
                    word[2 * e + 1] = qc::put_code(word[2 * e + 1], high_half(h[e]), inv, place);
                }
            }
            bytes[0] = __byte_perm(bytes[0], bytes[1], 0x5432);
            bytes[1] = __byte_perm(bytes[1], two[0] | two[1] << 8, 0x5432);
        }
        // the group's scale bytes, by its first lane
        if (o % 4 == 0) {
            uint8_t *sc = rec + R::kVScales + g * kQPage + p0 + 8 * q;
            if (lo <= 8 * q && hi >= 8 * q + 8) {
                *reinterpret_cast<uint2 *>(sc) = make_uint2(bytes[0], bytes[1]);
            } else {
#pragma unroll 1
                for (int u = max(lo - 8 * q, 0); u < min(hi - 8 * q, 8); ++u)
                    sc[u] = (uint8_t)((u < 4 ? bytes[0] : bytes[1]) >> (8 * (u % 4)));
            }
        }
    }
    if (lo >= hi) return;
    const uint32_t mask0 = code_mask(lo, hi), mask1 = code_mask(lo - 8, hi - 8);
    uint32_t *dst = reinterpret_cast<uint32_t *>(rec + R::kVCodes + ((p0 / 32) * D + 8 * o) * 16 +
                                                 p0 % 32 / 8 * 4);
    if ((mask0 & mask1) != 0xffffffffu) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint2 old = *reinterpret_cast<const uint2 *>(dst + 4 * c);
            first[c] = (first[c] & mask0) | (old.x & ~mask0);
            word[c] = (word[c] & mask1) | (old.y & ~mask1);
        }
    }
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint2 *>(dst + 4 * c) = make_uint2(first[c], word[c]);
}

// One warp per part of K or V of a (block, head): half a page (of V at D = 64: all of it).
//
// 65536 rows of 8 heads x 128 channels: 72.5 us for the 268 MB read and the 71 MB written,
// 4.7 TB/s, 70 % of the copy bandwidth.  Instructions bound it (issue slots 70 %, arithmetic
// pipe 54 %: some 120 per 8 channels of a row, of which 8 multiply-adds place codes; with
// shift and mask in their place 79 us), with the copies' latency beside them: eight CTAs of
// four warps per SM (16 pieces in flight per lane and six CTAs: 10 us more).  A warp per whole
// page of K or V took 106 us, a thread per group of channels 330.
template <int D>
__global__ void __launch_bounds__(kThreadsQ, kWriteCtas) qcache_write_kernel(const QRowsArgs a) {
    constexpr int kParts = 2, kVParts = D / 64;
    __shared__ uint4 s_stage[kThreadsQ / 32][kStage][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const Staged stage{s_stage[warp][0], lane};
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
        put_k<D>(rec, stage, off, warp * half, min(r.cnt, (warp + 1) * half),
                 static_cast<const __nv_bfloat16 *>(a.k), row);
    } else if (warp < kParts + kVParts) {
        put_v<D>(rec, stage, warp - kParts, off, r.cnt, static_cast<const __nv_bfloat16 *>(a.v),
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
// dependent loads, then the rows): with the positions read back 12.4 us for 16 requests, 46
// for 128 requests of 64-node trees.  Everything that reads
// ctx_len has read it before the barrier.  A warp per K, or part of V, of a head, in turn: 24
// of them while every request has an SM to itself (8 heads of 128 channels; 16 warps, and two
// rounds, for 16, 77 and 152 requests 3, 2.5 and 2.6 us longer), 16 beyond, when two CTAs
// share an SM (304 requests 51.8 to 48.8 us, 1000 requests 148 to 135).
constexpr int kThreadsCommit = 768, kThreadsMany = 512;

template <int D, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == kThreadsMany ? 2 : 1)
    qcache_commit_kernel(const QCommitArgs a) {
    extern __shared__ uint4 s_stage[];  // [warps][kStage][32]
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
    const Staged stage{s_stage + warp * kStage * 32, lane};
    constexpr int kTasks = 1 + D / 64;  // K, and the parts of V
    for (int u = warp; u < a.Hkv * kTasks; u += kThreads / 32) {
        const int h = u / kTasks, part = u % kTasks - 1;
        for (int m0 = 0; m0 < L;) {  // the pages that the path touches: one or two
            const int pos = ctx + m0, cnt = min(L - m0, kQPage - pos % kQPage);
            uint8_t *rec = a.cache +
                           ((size_t)s_page[pos / kQPage - ctx / kQPage] * a.Hkv + h) *
                               qc::Rec<D>::kBytes;
            auto row = [&](int m) { return (size_t)s_node[m0 + m] * a.stride + (size_t)h * D; };
            if (part < 0)
                put_k<D>(rec, stage, pos % kQPage, 0, cnt, static_cast<const __nv_bfloat16 *>(a.k),
                         row);
            else
                put_v<D>(rec, stage, part, pos % kQPage, cnt,
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

template <int D, int kThreads>
static cudaError_t launch_commit(const QCommitArgs &a, cudaStream_t s) {
    const cudaError_t e = configure_smem_once(qcache_commit_kernel<D, kThreads>, false);
    if (e != cudaSuccess) return e;
    return launch_pdl(qcache_commit_kernel<D, kThreads>, dim3(a.B), dim3(kThreads),
                      kThreads * kStage * sizeof(uint4), s, a);
}

template <int D>
static cudaError_t launch_commit_width(const QCommitArgs &a, cudaStream_t s) {
    return a.B > device_sms() ? launch_commit<D, kThreadsMany>(a, s)
                              : launch_commit<D, kThreadsCommit>(a, s);
}

cudaError_t launch_qcache_commit(const QCommitArgs &a, cudaStream_t s) {
    return a.d == 64 ? launch_commit_width<64>(a, s) : launch_commit_width<128>(a, s);
}

}  // namespace tv
