// prefill_tc.cu -- prompts through the gated linear recurrence on tensor cores: chunks of 64
// rows, one (request, head) per CTA at a time.
//
// With L_i the sum of the (log2) decays of a chunk up to row i, d = L_64 and H the state before
// the chunk:
//   O = diag(2^L) Q H + P V,       P_ij = 2^{L_i - L_j} q_i . k_j for j <= i, else 0
//   H' = 2^d H + (diag(2^{d - L}) K)^T V
// (Bole summary page, "Core techniques" §1, over a chain instead of a tree.)
//
// Everything that follows the state is transposed, so that the state's columns (dv) are the
// tensor memory's lanes:
//   S     = Q K^T           64 x 64     operands in shared memory
//   O1^T  = V^T P^T         dv x 64     V as it lies (MN-major), P's parts in shared memory
//   O2^T  = H^T Q^T         dv x 64     H's parts in tensor memory, Q as it lies
//   D^T   = V^T K~          dv x dk     V as it lies, K~ = diag(2^{d - L}) K in three parts
// H itself stays in the registers of sixteen warps (a lane per dv, dk / 4 channels a warp):
// H = 2^d H + D rounds once a chunk and to nearest, which the tensor cores' accumulation does
// not, and the next chunk's D can start as soon as this one's has been read.
//
// Precision.  P and H enter their products as NP bf16 parts, two for bf16 outputs (2^-16, far
// below the output's own rounding) and three for fp32; K~ always as three, since the state is
// fp32.  Small parts are accumulated first.  Decays are 64-bit fixed-point sums of log2 units
// (2^-32): differences of sums over a chunk lose nothing.  P's factor is 2^{L_i - R} 2^{R - L_j}
// around the middle R of the chunk's range, or, where a chunk spans more than 2^120, the
// exponential of each difference.
//
// Roles (32 warps): plan and decays (1), copies (1), products (1), K~ (6), H (16), outputs (4),
// P (3).
//
// Few long prompts: the rows of a request are cut into segments.  A first launch computes what
// each segment adds to a zero state, a second chains these sums, and the segments then run at
// the same time, each from its own state.
#include <type_traits>

#include "recurrence.cuh"
#include "tc_common.cuh"

namespace tv {
namespace {

constexpr int kC = 64;        // rows per chunk
constexpr int kStages = 3;    // chunks of q, k, v in flight
constexpr int kSlots = 4;     // chunks whose decays are ready
constexpr int kWarps = 32;
constexpr int kKeyWarps = 6, kScoreWarps = 3;  // of K~ and of P
constexpr int kThreadsT = kWarps * 32;
constexpr int kWaitTries = 1 << 20;  // 7800 cycles each at most: some 4 s
constexpr uint32_t kSlab = kC * 128; // 64 rows of 64 channels

enum { kA, kB, kW, kE };  // Slot::factor
enum Flags { kFirst = 1, kLast = 2, kEnd = 4, kMild = 8 };

struct alignas(16) Slot {
    float factor[4][kC];  // 2^{L - R}, 2^{R - L}, 2^{d - L}, 2^L
    long long L[kC];
    float2 d;             // 2^d as a pair
    int row, cnt, flags, head;
    long long src, dst;   // states: a (request, head), or ~index of one in the workspace
};

struct TcParams {
    PrefillArgs a;
    int seg;        // rows per segment, a multiple of kC
    int pieces;     // segments of a request of max_rows rows
    float *states;  // [B][pieces][H][dk][dv]: the state before each segment
    float2 *decays; // [B][pieces][H]
    int expire;     // test hook: leave the first chunk's copies out
};

template <int DK, int DV, int NP>
struct Lay {
    static constexpr uint32_t kQ = 0, kK = DK * 128, kV = 2 * DK * 128,
                              kStage = (2 * DK + DV) * 128;
    static constexpr uint32_t kKt = kStages * kStage, kKtPart = DK * 128;
    static constexpr uint32_t kP = kKt + 3 * kKtPart, kPPart = kC * 128;
    static constexpr uint32_t kSlot0 = kP + NP * kPPart;
    static constexpr uint32_t kBytes = kSlot0 + kSlots * (uint32_t)sizeof(Slot) + 1024;
    // tensor memory columns
    static constexpr uint32_t tD = 0, tH = DK, tS = tH + NP * DK / 2, tO1 = tS + kC,
                              tO2 = tO1 + kC, kCols = 512;
    static_assert(tO2 + kC <= kCols, "tensor memory");
    static_assert(kBytes <= tcc::kSmemLimit - 512, "shared memory");
};

// Two floats in a register pair, for the packed fp32 instructions.
__device__ __forceinline__ uint64_t two(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint64_t two(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ void halves(uint64_t x, uint32_t &lo, uint32_t &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A pair as NP packed pairs of bf16 parts: upper bits cut off, the last part rounded.
template <int NP>
__device__ __forceinline__ void split_pair(uint64_t x, uint32_t (&part)[NP]) {
    uint32_t b0, b1;
#pragma unroll
    for (int p = 0; p + 1 < NP; ++p) {
        halves(x, b0, b1);
        part[p] = __byte_perm(b0, b1, 0x7632);
        x = sub2(x, two(b0 & 0xFFFF0000u, b1 & 0xFFFF0000u));
    }
    halves(x, b0, b1);
    const __nv_bfloat162 l = __floats2bfloat162_rn(__uint_as_float(b0), __uint_as_float(b1));
    part[NP - 1] = *reinterpret_cast<const uint32_t *>(&l);
}

// 2^(x 2^-32).
__device__ __forceinline__ rec::Pair exp2_fixed(long long x) {
    const long long n = (x + (1LL << 31)) >> 32;
    const float f = (float)(int32_t)(x - (n << 32)) * 2.3283064365386963e-10f;
    return rec::exp2_pair((float)(int)max(min(n, 4096LL), -4096LL), f);
}
// The same as one float, by the hardware's exponential (2^-22) of the fraction.
__device__ __forceinline__ float exp2_single(long long x) {
    const long long n = (x + (1LL << 31)) >> 32;
    const float f = (float)(int32_t)(x - (n << 32)) * 2.3283064365386963e-10f;
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(f));
    return e * __int_as_float(((int)max(min(n, 128LL), -127LL) + 127) << 23);
}

// A CTA's walk over its chunks.  An item is a segment of a request and head; a CTA begins with
// the item of its block index and then takes over items of CTAs that have not been launched, so
// that long and short ones even out.
struct Walk {
    int item;              // (b * pieces + segment) * H + head, without the last segments if !OUT
    int asked;             // items asked for so far
    int row, end, head;    // of the current item; row >= end: none left of it
    bool first, done;
    long long unit, ws;    // b * H + head, and the segment's place in the workspace
    int piece, pieces;     // its number, and the request's segments
};

template <int DK, int DV, int NP, bool OUT>
__global__ void __launch_bounds__(kThreadsT, 1)
    prefill_tc_kernel(const __grid_constant__ CUtensorMap map_q,
                      const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v, const TcParams p) {
    using L = Lay<DK, DV, NP>;
    constexpr int kQuads = DV / 32;           // quadrants of lanes that hold something
    constexpr int kChan = DK / 4;             // channels of a lane of the H warps
    extern __shared__ uint8_t s_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ __align__(8) uint64_t s_gate_full[kSlots], s_gate_free[kSlots], s_full[kStages],
        s_empty[kStages], s_s_full, s_p_full, s_kt_full, s_h_full, s_kv_done, s_o_full, s_o_free, s_drain, s_asked;
    __shared__ __align__(16) uint64_t s_answer[2];
    const PrefillArgs &a = p.a;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    uint8_t *s_base = s_raw + ((1024 - (ptx::smem_addr(s_raw) & 1023)) & 1023);
    const uint32_t base = ptx::smem_addr(s_base);
    Slot *slots = reinterpret_cast<Slot *>(s_base + L::kSlot0);

    const auto bar = [](const uint64_t &b) { return ptx::smem_addr(&b); };
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < kSlots; ++i) {
            ptx::mbar_init(bar(s_gate_full[i]), 1);
            // readers: copies, products, K~, H and, with outputs, the outputs' and P's warps
            ptx::mbar_init(bar(s_gate_free[i]),
                           2 + kKeyWarps + 4 * kQuads + (OUT ? kQuads + kScoreWarps : 0));
        }
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(bar(s_full[i]), 1);
            ptx::mbar_init(bar(s_empty[i]), 1);
        }
        ptx::mbar_init(bar(s_s_full), 1);
        ptx::mbar_init(bar(s_p_full), kScoreWarps);
        ptx::mbar_init(bar(s_kt_full), kKeyWarps);
        ptx::mbar_init(bar(s_h_full), 4 * kQuads);
        ptx::mbar_init(bar(s_kv_done), 1);
        ptx::mbar_init(bar(s_o_full), 1);
        ptx::mbar_init(bar(s_o_free), kQuads);
        ptx::mbar_init(bar(s_drain), 1);
        ptx::mbar_init(bar(s_asked), 1);
        ptx::fence_mbar_init();
        if (OUT) ptx::prefetch_tensormap(&map_q);
        ptx::prefetch_tensormap(&map_k);
        ptx::prefetch_tensormap(&map_v);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_addr(&s_tmem), L::kCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = s_tmem;
    pdl_wait();
    pdl_launch_next();

    // A wait that expires raises the CTA's flag; its warp leaves, and the others' waits end early.
    const int tries = p.expire ? kWaitTries / 64 : kWaitTries;
    const auto wait = [&](const uint64_t &b, uint32_t parity) {
        bool ok = ptx::mbar_wait_tries(bar(b), parity, 16);
        for (int i = 16; !ok && i < tries && *(volatile int *)&s_abort == 0; i += 64)
            ok = ptx::mbar_wait_tries(bar(b), parity, 64);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && lane == 0) *(volatile int *)&s_abort = 1;
        return ok;
    };
    const auto arrive = [&](const uint64_t &b) {  // once per warp, after all of its lanes
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(b));
    };
    // the slot of chunk n, once its decays are there
    const auto gate = [&](int n, Slot *&s) {
        s = slots + n % kSlots;
        return wait(s_gate_full[n % kSlots], (n / kSlots) & 1);
    };

    if (warp == 0) {
        // ---- plan, copies, decays
        Walk w{};
        const int per = OUT ? p.pieces : p.pieces - 1;
        const auto ask = [&]() {
            if (lane == 0) {
                ptx::fence_proxy_async_smem();  // (the answer before has been read)
                ptx::mbar_arrive_expect_tx(bar(s_asked), 16);
                ptx::try_cancel(ptx::smem_addr(s_answer), bar(s_asked));
            }
            __syncwarp();
            ++w.asked;
        };
        const auto next_item = [&](bool begin) {
            for (;; begin = false) {
                if (begin) {
                    w.item = blockIdx.x;
                } else {
                    if (!wait(s_asked, (w.asked - 1) & 1)) {
                        w.done = true;
                        return;
                    }
                    w.item = ptx::cancelled_cta(ptx::smem_addr(s_answer));
                    __syncwarp();
                    if (w.item < 0) {
                        w.done = true;
                        return;
                    }
                }
                ask();
                const int slot = w.item / a.H, b = slot / per, i = slot - b * per;
                int off, n;
                if (!request_range(a.offsets, b, a.R, a.max_rows, off, n)) {
                    if (lane == 0) report(a.status, TV_ERR_TREE);
                    continue;
                }
                const int pieces = max(1, (n + p.seg - 1) / p.seg);
                if (i >= pieces || (!OUT && i == pieces - 1)) continue;
                w.head = w.item - slot * a.H;
                w.row = off + i * p.seg;
                w.end = w.row + min(p.seg, n - i * p.seg);
                w.first = true;
                w.unit = (long long)b * a.H + w.head;
                w.ws = ((long long)b * p.pieces + i) * a.H + w.head;
                w.piece = i;
                w.pieces = pieces;
                return;
            }
        };
        next_item(true);
        float g0 = 0.f, g1 = 0.f;
        const auto fetch = [&](const Walk &at) {  // the decays of the chunk at w
            const int t = at.row + 2 * lane, cnt = at.done ? 0 : min(kC, at.end - at.row);
            const float *g = a.g + at.head;
            g0 = 2 * lane < cnt ? g[(size_t)t * a.g_stride] : 0.f;
            g1 = 2 * lane + 1 < cnt ? g[((size_t)t + 1) * a.g_stride] : 0.f;
        };
        fetch(w);
        long long total = 0;  // log2 of the item's decay so far
        bool total_nan = false;
        for (int n = 0;; ++n) {
            Slot *s = slots + n % kSlots;
            if (n >= kSlots && !wait(s_gate_free[n % kSlots], ((n / kSlots) & 1) ^ 1)) break;
            if (w.done) {
                if (lane == 0) s->flags = kEnd;
                arrive(s_gate_full[n % kSlots]);
                break;
            }
            if (p.expire) {
                wait(s_asked, (w.asked - 1) & 1);
                break;
            }
            const int row = w.row, cnt = min(kC, w.end - row), head = w.head;
            const bool first = w.first, last = row + kC >= w.end;
            const Walk now = w;
            const float x0 = g0, x1 = g1;
            w.first = false;
            w.row += kC;
            if (last) next_item(false);
            fetch(w);  // the next chunk's, on its way while this one's are summed

            const float most = 2839.f;  // 4096 log2 units
            const bool nan0 = x0 != x0, nan1 = x1 != x1;
            const double unit = 1.4426950408889634 * 4294967296.0;
            const long long y0 = nan0 ? 0 : __double2ll_rn((double)fminf(fmaxf(x0, -most), most) * unit);
            const long long y1 = nan1 ? 0 : __double2ll_rn((double)fminf(fmaxf(x1, -most), most) * unit);
            long long sum = y0 + y1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            const long long l0 = sum - y1, l1 = sum, end = __shfl_sync(0xffffffffu, sum, 31);
            const int h0 = (int)(l0 >> 32), h1 = (int)(l1 >> 32);
            const int lo = __reduce_min_sync(0xffffffffu, min(h0, h1));
            const int hi = __reduce_max_sync(0xffffffffu, max(h0, h1));
            const bool mild = hi - lo <= 120;
            const long long mid = (long long)((lo + hi) / 2) * (1LL << 32);
            // from the first NaN on, everything of this request and head is one
            const uint32_t bad0 = __ballot_sync(0xffffffffu, nan0),
                           bad1 = __ballot_sync(0xffffffffu, nan1);
            const bool any = (bad0 | bad1) != 0;
            const uint32_t upto = 0xffffffffu >> (31 - lane);
            const bool n0 = (bad0 & upto) || (bad1 & (upto >> 1)), n1 = ((bad0 | bad1) & upto) != 0;
            const float nanf = __int_as_float(0x7fffffff);
            if (!mild) {
                s->L[2 * lane] = l0;
                s->L[2 * lane + 1] = l1;
            }
            // a, b, w, e: 2^{L - R}, 2^{R - L}, 2^{d - L}, 2^L (a and b are 1 where R will not do)
            const long long zero = mild ? mid : 0;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                const long long from = c == 3 ? 0 : c == 2 ? end : zero;
                long long z0 = l0 - from, z1 = l1 - from;
                if (c == 1 || c == 2) {
                    z0 = -z0;
                    z1 = -z1;
                }
                if (c < 2 && !mild) z0 = z1 = 0;
                float2 f = make_float2(exp2_single(z0), exp2_single(z1));
                if (c == 0 || c == 3) {
                    if (n0) f.x = nanf;
                    if (n1) f.y = nanf;
                }
                *reinterpret_cast<float2 *>(s->factor[c] + 2 * lane) = f;
            }
            if (first) {
                total = 0;
                total_nan = false;
            }
            total += end;
            total_nan |= any;
            if (lane == 0) {
                const rec::Pair d = exp2_fixed(end);
                s->d = any ? make_float2(nanf, nanf) : make_float2(d.hi, d.lo);
                s->row = row;
                s->cnt = cnt;
                s->head = head;
                s->flags = (first ? kFirst : 0) | (last ? kLast : 0) | (mild ? kMild : 0);
                if (OUT) {
                    s->src = now.pieces > 1 ? ~now.ws : now.unit;
                    s->dst = now.piece == now.pieces - 1 ? now.unit : -1;
                } else {
                    s->src = -1;
                    s->dst = ~(now.ws + a.H);  // where the next segment begins
                    if (last) {
                        const rec::Pair t = exp2_fixed(total);
                        p.decays[now.ws] = total_nan ? make_float2(nanf, nanf)
                                                     : make_float2(t.hi, t.lo);
                    }
                }
            }
            arrive(s_gate_full[n % kSlots]);
        }
    } else if (warp == 2) {
        // ---- copies
        int issued = 0;
        for (int n = 0;; ++n) {
            Slot *s;
            if (!gate(n, s)) break;
            if (s->flags & kEnd) break;
            // a stage is free once every product of the chunk before in it is done
            if (n >= kStages && !wait(s_empty[n % kStages], ((n / kStages) & 1) ^ 1)) break;
            if (lane == 0) {
                const int head = s->head, row = s->row;
                const uint32_t at = base + n % kStages * L::kStage, full = bar(s_full[n % kStages]);
                ptx::mbar_arrive_expect_tx(full, OUT ? L::kStage : L::kStage - L::kK);
                for (int c = 0; c < DK / 64; ++c) {
                    if (OUT)
                        ptx::tma_load_3d(at + L::kQ + c * kSlab, &map_q, c * 64, head, row, full);
                    ptx::tma_load_3d(at + L::kK + c * kSlab, &map_k, c * 64, head, row, full);
                }
                for (int c = 0; c < DV / 64; ++c)
                    ptx::tma_load_3d(at + L::kV + c * kSlab, &map_v, c * 64, head, row, full);
            }
            issued = n + 1;
            arrive(s_gate_free[n % kSlots]);
        }
        // copies that nobody waited for (after a timeout)
        if (*(volatile int *)&s_abort)
            for (int i = max(0, issued - kStages); i < issued; ++i)
                ptx::mbar_wait_tries(bar(s_full[i % kStages]), (i / kStages) & 1, 1 << 14);
    } else if (warp == 1) {
        // ---- products
        const uint32_t lead = ptx::elect_one();
        const auto stage = [&](int n) { return base + n % kStages * L::kStage; };
        // descriptors move by their address field, in units of 16 bytes
        const auto scores = [&](int n) {
            // 128 lanes take the 64 rows behind the tile along; nobody reads their results
            const uint64_t q = ptx::desc_kmajor_sw128(stage(n) + L::kQ, 1024),
                           k = ptx::desc_kmajor_sw128(stage(n) + L::kK, 1024);
#pragma unroll
            for (int kk = 0; kk < DK / 16; ++kk) {
                const uint32_t o = (kk / 4 * kSlab + kk % 4 * 32) / 16;
                ptx::mma_bf16_lead(tmem + L::tS, q + o, k + o, ptx::idesc_bf16_f32(128, kC), kk > 0,
                                   lead);
            }
            ptx::mma_commit_lead(bar(s_s_full), lead);
        };
        // (the flags by a reduction, so that the flow is known to be the whole warp's and the
        // products' operands stay in uniform registers)
        const auto more = [&](int n) {
            Slot *s;
            return gate(n, s) && !(__reduce_or_sync(0xffffffffu, s->flags) & kEnd);
        };
        bool ok = more(0);
        if (ok && OUT) {
            ok = wait(s_full[0], 0);
            ptx::tc_fence_after_sync();
            if (ok) scores(0);
        }
        for (int n = 0; ok; ++n) {
            const uint32_t ph = n & 1, q = stage(n) + L::kQ, v = stage(n) + L::kV;
            if (!OUT && !(ok = wait(s_full[n % kStages], (n / kStages) & 1))) break;
            if (OUT && n > 0 && !(ok = wait(s_o_free, ph ^ 1))) break;
            if (!(ok = wait(s_h_full, ph))) break;
            ptx::tc_fence_after_sync();
            const uint64_t vd = ptx::desc_mnmajor_sw128(v, kSlab, 1024);
            if (OUT) {
                const uint64_t qd = ptx::desc_kmajor_sw128(q, 1024);
#pragma unroll 1
                for (int part = NP - 1; part >= 0; --part)
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk)
                        ptx::mma_bf16_ts_lead(
                            tmem + L::tO2, tmem + L::tH + part * (DK / 2) + kk * 8,
                            qd + (kk / 4 * kSlab + kk % 4 * 32) / 16,
                            ptx::idesc_bf16_f32(128, kC), part < NP - 1 || kk > 0, lead);
            }
            if (!(ok = wait(s_kt_full, ph))) break;
            ptx::tc_fence_after_sync();
#pragma unroll 1
            for (int part = 2; part >= 0; --part) {
                const uint64_t kd =
                    ptx::desc_mnmajor_sw128(base + L::kKt + part * L::kKtPart, kSlab, 1024);
#pragma unroll
                for (int kk = 0; kk < kC / 16; ++kk)
                    ptx::mma_bf16_lead(tmem + L::tD, vd + kk * 128, kd + kk * 128,
                                       ptx::idesc_bf16_f32_abmn(128, DK), part < 2 || kk > 0, lead);
            }
            ptx::mma_commit_lead(bar(s_kv_done), lead);
            if (OUT) {
                if (!(ok = wait(s_p_full, ph))) break;
                ptx::tc_fence_after_sync();
#pragma unroll 1
                for (int part = NP - 1; part >= 0; --part) {
                    const uint64_t pd =
                        ptx::desc_kmajor_sw128(base + L::kP + part * L::kPPart, 1024);
#pragma unroll
                    for (int kk = 0; kk < kC / 16; ++kk)
                        ptx::mma_bf16_lead(tmem + L::tO1, vd + kk * 128, pd + kk * 2,
                                           ptx::idesc_bf16_f32_amn(128, kC), part < NP - 1 || kk > 0,
                                           lead);
                }
                ptx::mma_commit_lead(bar(s_o_full), lead);
            }
            ptx::mma_commit_lead(bar(s_empty[n % kStages]), lead);
            arrive(s_gate_free[n % kSlots]);
            if (!(ok = more(n + 1))) break;
            if (OUT) {
                // (P of chunk n has been written, so its scores have been read)
                if (!(ok = wait(s_full[(n + 1) % kStages], ((n + 1) / kStages) & 1))) break;
                ptx::tc_fence_after_sync();
                scores(n + 1);
            }
        }
        ptx::mma_commit_lead(bar(s_drain), lead);
        __syncwarp();
        ptx::mbar_wait_tries(bar(s_drain), 0, 1 << 18);
    } else if (warp == 3 || (warp >= 26 && warp != 29)) {
        // ---- K~: keys times 2^{d - L}, in three parts, laid out as the keys are
        const int t = (warp == 3 ? 0 : warp < 29 ? warp - 25 : warp - 26) * 32 + lane;
        for (int n = 0;; ++n) {
            Slot *s;
            if (!gate(n, s)) break;
            if (s->flags & kEnd) break;
            if (!wait(s_full[n % kStages], (n / kStages) & 1)) break;
            if (n > 0 && !wait(s_kv_done, (n & 1) ^ 1)) break;
            uint8_t *st = s_base + n % kStages * L::kStage;
            const int cnt = s->cnt;
            if (cnt < kC) {  // rows past the segment belong to others: they may hold anything
                for (int i = t; i < (kC - cnt) * (DV / 8); i += kKeyWarps * 32) {
                    const int r = cnt + i / (DV / 8), c = i % (DV / 8);
                    *reinterpret_cast<uint4 *>(st + L::kV + c / 8 * kSlab + r * 128 + c % 8 * 16) =
                        make_uint4(0, 0, 0, 0);
                }
            }
#pragma unroll 2
            for (int at = t * 16; at < DK * 128; at += kKeyWarps * 32 * 16) {
                const int r = at / 128 % kC;
                uint4 x = *reinterpret_cast<const uint4 *>(st + L::kK + at);
                if (r >= cnt) x = make_uint4(0, 0, 0, 0);
                const float w = s->factor[kW][r];
                const uint64_t w2 = two(w, w);
                const uint32_t in[4] = {x.x, x.y, x.z, x.w};
                uint32_t out[3][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t part[3];
                    split_pair<3>(mul2(two(in[e] << 16, in[e] & 0xFFFF0000u), w2), part);
#pragma unroll
                    for (int j = 0; j < 3; ++j) out[j][e] = part[j];
                }
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    *reinterpret_cast<uint4 *>(s_base + L::kKt + j * L::kKtPart + at) =
                        make_uint4(out[j][0], out[j][1], out[j][2], out[j][3]);
            }
            ptx::fence_proxy_async_smem();
            arrive(s_kt_full);
            arrive(s_gate_free[n % kSlots]);
        }
    } else if (warp < 20) {
        // ---- H: lane = column of the state, kChan of its channels in registers
        const int quad = warp % 4, c0 = (warp - 4) / 4 * kChan, col = quad * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)quad << 21);  // lane quad * 32
        if (quad < kQuads) {
            uint64_t h[kChan / 2];
            for (int n = 0;; ++n) {
                Slot *s;
                if (!gate(n, s)) break;
                const int flags = s->flags;
                if (flags & kEnd) break;
                if (flags & kFirst) {
                    const long long src = s->src;
                    const float *from = !OUT       ? nullptr
                                        : src < 0  ? p.states + (size_t)~src * DK * DV
                                        : a.H0     ? a.H0 + (size_t)src * DK * DV
                                                   : nullptr;
#pragma unroll
                    for (int i = 0; i < kChan / 2; ++i)
                        h[i] = from ? two(from[(c0 + 2 * i) * DV + col],
                                          from[(c0 + 2 * i + 1) * DV + col])
                                    : 0;
                }
                if (OUT) {
#pragma unroll
                    for (int i0 = 0; i0 < kChan / 2; i0 += 8) {
                        uint32_t part[NP][8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            uint32_t x[NP];
                            split_pair<NP>(h[i0 + i], x);
#pragma unroll
                            for (int j = 0; j < NP; ++j) part[j][i] = x[j];
                        }
#pragma unroll
                        for (int j = 0; j < NP; ++j)
                            ptx::tmem_st_x8(lanes + L::tH + j * (DK / 2) + c0 / 2 + i0, part[j]);
                    }
                    ptx::tmem_wait_st();
                }
                ptx::tc_fence_before_sync();
                arrive(s_h_full);
                const uint64_t dx = two(s->d.x, s->d.x), dy = two(s->d.y, s->d.y);
                const long long dst = s->dst;
                arrive(s_gate_free[n % kSlots]);
                if (!wait(s_kv_done, n & 1)) break;
                ptx::tc_fence_after_sync();
#pragma unroll
                for (int i0 = 0; i0 < kChan; i0 += 16) {
                    uint32_t x[16];
                    ptx::tmem_ld_x16_nowait(lanes + L::tD + c0 + i0, x);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint64_t &y = h[i0 / 2 + i];
                        y = fma2(y, dx, fma2(y, dy, two(x[2 * i], x[2 * i + 1])));
                    }
                }
                if ((flags & kLast) && (!OUT || dst >= 0)) {
                    float *to = dst < 0 ? p.states + (size_t)~dst * DK * DV
                                        : a.H_new + (size_t)dst * DK * DV;
#pragma unroll
                    for (int i = 0; i < kChan / 2; ++i) {
                        uint32_t x, y;
                        halves(h[i], x, y);
                        to[(c0 + 2 * i) * DV + col] = __uint_as_float(x);
                        to[(c0 + 2 * i + 1) * DV + col] = __uint_as_float(y);
                    }
                }
            }
        }
    } else if (warp < 24) {
        // ---- outputs: lane = column, 64 rows
        const int quad = warp % 4, col = quad * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)quad << 21);
        if (OUT && quad < kQuads) {
            for (int n = 0;; ++n) {
                Slot *s;
                if (!gate(n, s)) break;
                if (s->flags & kEnd) break;
                const int cnt = s->cnt;
                using O = std::conditional_t<NP == 3, float, __nv_bfloat16>;
                const size_t step = (size_t)a.H * DV;
                O *to = static_cast<O *>(a.out) + s->row * step + s->head * DV + col;
                if (!wait(s_o_full, n & 1)) break;
                ptx::tc_fence_after_sync();
#pragma unroll 1
                for (int t0 = 0; t0 < kC; t0 += 16) {
                    uint32_t x[16], y[16];
                    ptx::tmem_ld_x16_nowait(lanes + L::tO1 + t0, x);
                    ptx::tmem_ld_x16_nowait(lanes + L::tO2 + t0, y);
                    ptx::tmem_wait_ld();
                    if (t0 == kC - 16) {
                        ptx::tc_fence_before_sync();
                        arrive(s_o_free);
                    }
                    const float4 *e4 = reinterpret_cast<const float4 *>(s->factor[kE] + t0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 f = e4[i];
                        uint32_t o[4];
                        halves(fma2(two(f.x, f.y), two(y[4 * i], y[4 * i + 1]),
                                    two(x[4 * i], x[4 * i + 1])), o[0], o[1]);
                        halves(fma2(two(f.z, f.w), two(y[4 * i + 2], y[4 * i + 3]),
                                    two(x[4 * i + 2], x[4 * i + 3])), o[2], o[3]);
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            if (t0 + 4 * i + u < cnt) *to = O(__uint_as_float(o[u]));
                            to += step;
                        }
                    }
                }
                arrive(s_gate_free[n % kSlots]);
            }
        }
    } else {
        // ---- P: lane = row of the chunk; two blocks of 16 columns each for warp 24 (rows 0-31,
        // which reach no further), 25 and 29 (rows 32-63)
        if (OUT) {
            const int quad = warp % 4, i = quad * 32 + lane, from = warp == 29 ? 2 : 0;
            const uint32_t lanes = tmem + ((uint32_t)quad << 21);
            uint8_t *row = s_base + L::kP + i * 128;
            if (warp == 24)  // zero once and for all: columns past the rows
                for (int c = 4; c < 8; ++c)
                    for (int j = 0; j < NP; ++j)
                        *reinterpret_cast<uint4 *>(row + j * L::kPPart + ((c ^ (i & 7)) * 16)) =
                            make_uint4(0, 0, 0, 0);
            for (int n = 0;; ++n) {
                Slot *s;
                if (!gate(n, s)) break;
                const int flags = s->flags;
                if (flags & kEnd) break;
                if (!wait(s_s_full, n & 1)) break;
                if (n > 0 && !wait(s_o_full, (n & 1) ^ 1)) break;  // P of the chunk before is read
                ptx::tc_fence_after_sync();
                const float ai = s->factor[kA][i];
                const uint64_t a2 = two(ai, ai);
#pragma unroll 1
                for (int jb = from; jb < from + 2; ++jb) {
                    uint32_t x[16];
                    uint64_t f[8];
                    ptx::tmem_ld_x16_nowait(lanes + L::tS + jb * 16, x);
                    if (flags & kMild) {
                        const float4 *b4 = reinterpret_cast<const float4 *>(s->factor[kB] + jb * 16);
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float4 b = b4[u];
                            f[2 * u] = mul2(a2, two(b.x, b.y));
                            f[2 * u + 1] = mul2(a2, two(b.z, b.w));
                        }
                    } else {
                        // decays that span too much for factors around a middle (rare)
                        const long long Li = s->L[i];
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const int j = jb * 16 + 2 * u;
                            f[u] = mul2(a2, two(exp2_single(Li - s->L[j]),
                                                exp2_single(Li - s->L[j + 1])));
                        }
                    }
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t out[NP][4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int u = 4 * c + e, j = jb * 16 + 2 * u;
                            uint32_t y0, y1, part[NP];
                            halves(mul2(two(x[2 * u], x[2 * u + 1]), f[u]), y0, y1);
                            split_pair<NP>(two(j <= i ? y0 : 0u, j < i ? y1 : 0u), part);
#pragma unroll
                            for (int q = 0; q < NP; ++q) out[q][e] = part[q];
                        }
                        uint8_t *at = row + (((jb * 2 + c) ^ (i & 7)) * 16);
#pragma unroll
                        for (int q = 0; q < NP; ++q)
                            *reinterpret_cast<uint4 *>(at + q * L::kPPart) =
                                make_uint4(out[q][0], out[q][1], out[q][2], out[q][3]);
                    }
                }
                ptx::tc_fence_before_sync();
                ptx::fence_proxy_async_smem();
                arrive(s_p_full);
                arrive(s_gate_free[n % kSlots]);
            }
        }
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (tid == 0 && s_abort) report(a.status, TV_ERR_TIMEOUT);
    if (warp == 1) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, L::kCols);
    }
}

// The segments' states from what each adds: S_{i+1} = 2^{d_i} S_i + added_i.
constexpr int kThreadsChain = 256;
__global__ void __launch_bounds__(kThreadsChain) prefill_chain_kernel(TcParams p) {
    const PrefillArgs &a = p.a;
    const int unit = blockIdx.x, b = unit / a.H, h = unit % a.H;
    const size_t quads = (size_t)a.dk * a.dv / 4, at = (size_t)blockIdx.y * kThreadsChain + threadIdx.x;
    pdl_wait();
    pdl_launch_next();
    int off, n;
    if (at >= quads || !request_range(a.offsets, b, a.R, a.max_rows, off, n)) return;
    const int pieces = (n + p.seg - 1) / p.seg;
    if (pieces < 2) return;
    const size_t first = (size_t)b * p.pieces * a.H + h;
    float4 *state = reinterpret_cast<float4 *>(p.states) + first * quads + at;
    const float2 *decay = p.decays + first;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.H0) x = reinterpret_cast<const float4 *>(a.H0)[(size_t)unit * quads + at];
    *state = x;
    for (int i = 1; i < pieces; ++i) {
        const float2 d = decay[(size_t)(i - 1) * a.H];
        float4 &to = state[(size_t)i * a.H * quads];
        const float4 y = to;
        x.x = fmaf(x.x, d.x, fmaf(x.x, d.y, y.x));
        x.y = fmaf(x.y, d.x, fmaf(x.y, d.y, y.y));
        x.z = fmaf(x.z, d.x, fmaf(x.z, d.y, y.z));
        x.w = fmaf(x.w, d.x, fmaf(x.w, d.y, y.w));
        to = x;
    }
}

// ---------------------------------------------------------------- host side

// Pieces that a request of the bound's length is cut into: what makes the longest SM's work
// least, counted in chunks.  A segment costs a few chunks to start and its first launch about
// half of a chunk's work for each.
int best_pieces(const PrefillArgs &a) {
    const long long units = (long long)a.B * a.H, sms = device_sms();
    const long long chunks = (a.max_rows + kC - 1LL) / kC;
    const auto waves = [&](long long items) { return (double)((items + sms - 1) / sms); };
    int best = 1;
    double least = waves(units) * (chunks + 4.0);
    if (units > 8 * sms) return 1;
    for (int s = 2; s <= 64 && s <= chunks; ++s) {
        const double per = (double)((chunks + s - 1) / s);
        const double cost = waves(units * s) * (per + 4.0) + waves(units * (s - 1)) * (0.6 * per + 4.0) + 8.0;
        if (cost < 0.95 * least) {
            least = cost;
            best = s;
        }
    }
    return best;
}

int segment_rows(const PrefillArgs &a, int pieces) {
    const long long chunks = (a.max_rows + kC - 1LL) / kC;
    return (int)std::min<long long>((chunks + pieces - 1) / pieces * kC, 0x40000000);
}

size_t cut_bytes(const PrefillArgs &a, int pieces) {
    const size_t items = (size_t)a.B * pieces * a.H;
    return items * a.dk * a.dv * 4 + (items * 8 + 15) / 16 * 16;
}

bool rows_map(CUtensorMap *m, const void *base, int width, int H, int R, int64_t stride) {
    const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)H, (cuuint64_t)R};
    const cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, kC}, one[3] = {1, 1, 1};
    const auto encode = tcc::encode_fn();
    return encode && encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims,
                            strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV, int NP, bool OUT>
cudaError_t launch_kernel(const TcParams &p, const CUtensorMap *m, cudaStream_t s) {
    const cudaError_t e = configure_smem_once(prefill_tc_kernel<DK, DV, NP, OUT>, false);
    if (e != cudaSuccess) return e;
    const unsigned items = (unsigned)p.a.B * (OUT ? p.pieces : p.pieces - 1) * p.a.H;
    return launch_pdl(prefill_tc_kernel<DK, DV, NP, OUT>, dim3(items), dim3(kThreadsT),
                      Lay<DK, DV, NP>::kBytes, s, m[0], m[1], m[2], p);
}

template <int DK, int DV>
cudaError_t launch_widths(const PrefillArgs &a, bool expire, cudaStream_t s) {
    CUtensorMap m[3];
    if (!rows_map(&m[0], a.q, DK, a.H, a.R, a.q_stride) ||
        !rows_map(&m[1], a.k, DK, a.H, a.R, a.k_stride) ||
        !rows_map(&m[2], a.v, DV, a.H, a.R, a.v_stride))
        return cudaErrorInvalidValue;
    TcParams p{};
    p.a = a;
    p.expire = expire;
    int pieces = best_pieces(a);
    while (pieces > 1 && cut_bytes(a, pieces) > a.ws_bytes) --pieces;
    p.seg = segment_rows(a, pieces);
    p.pieces = pieces;
    if (pieces > 1) {
        p.states = reinterpret_cast<float *>(a.ws);
        p.decays = reinterpret_cast<float2 *>(a.ws + (size_t)a.B * pieces * a.H * DK * DV * 4);
        cudaError_t e = launch_kernel<DK, DV, 2, false>(p, m, s);
        if (e != cudaSuccess) return e;
        e = launch_pdl(prefill_chain_kernel,
                       dim3((unsigned)(a.B * a.H), (DK * DV / 4 + kThreadsChain - 1) / kThreadsChain),
                       dim3(kThreadsChain), 0, s, p);
        if (e != cudaSuccess) return e;
    }
    return a.out_f32 ? launch_kernel<DK, DV, 3, true>(p, m, s)
                     : launch_kernel<DK, DV, 2, true>(p, m, s);
}

}  // namespace

bool prefill_tc_supported(const PrefillArgs &a) {
    const int64_t most = 1LL << 38;  // a tensor map's strides are below 2^40 bytes
    return a.qkv_dtype == TV_BF16 && a.decay == TV_DECAY_SCALAR && (a.dk == 64 || a.dk == 128) &&
           (a.dv == 64 || a.dv == 128) && a.R > 0 && a.q_stride < most && a.k_stride < most &&
           a.v_stride < most;
}

size_t prefill_tc_workspace_bytes(const PrefillArgs &a) {
    const int pieces = best_pieces(a);
    return pieces > 1 ? cut_bytes(a, pieces) : 0;
}

cudaError_t launch_prefill_tc(const PrefillArgs &a, bool expire, cudaStream_t s) {
    if (a.dk == 64)
        return a.dv == 64 ? launch_widths<64, 64>(a, expire, s) : launch_widths<64, 128>(a, expire, s);
    return a.dv == 64 ? launch_widths<128, 64>(a, expire, s) : launch_widths<128, 128>(a, expire, s);
}

}  // namespace tv
