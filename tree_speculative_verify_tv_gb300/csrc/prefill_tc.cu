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
//   O2^T  = H^T Q^T         dv x 64     H's parts in tensor memory, Q as it lies; added to O1^T
//   D^T   = V^T K~          dv x dk     V as it lies, K~ = diag(2^{d - L}) K in three parts
// H itself stays in the registers of sixteen warps (a lane per dv, dk / 4 channels a warp):
// H = 2^d H + D rounds once a chunk and to nearest, which the tensor cores' accumulation does
// not, and the next chunk's D can start as soon as this one's has been read.
//
// O1 and O2 are summed in one accumulator: both carry the factor 2^{R - L} of the middle R of the
// chunk's range of L, and the output's 2^{L - R} comes last:
//   O = diag(2^{L - R}) (Q (2^R H) + P V),   P_ij = 2^{R - L_j} q_i . k_j
// A chunk ends early where L would span more than 2^120.
//
// Precision.  P and H enter their products as NP bf16 parts, two for bf16 outputs (2^-16, far
// below the output's own rounding) and three for fp32; K~ (or V~, see below) always as three,
// since the state is fp32.  Small parts are accumulated first.  Decays are 64-bit fixed-point sums
// of log2 units (2^-40, what a row's is cut to): differences of sums over a chunk lose nothing more.
// The factors 2^{R - L}, 2^{d - L} and 2^{L - R} come from the hardware's exponential (2^-22).
//
// The decays of D's product may stand with either factor: V~ = diag(2^{d - L}) V where dv is the
// smaller (half the conversions at dk = 128, dv = 64), else K~.
//
// Roles (32 warps): plan with the decays, and copies (one or two warps), D's product, the outputs'
// products (a warp each), K~ or V~ (4 to 8), H (16), outputs (4), P (3).  D waits for nothing but
// H's sums of the chunk before, so that parts, outputs and scores stay off the chain from chunk to
// chunk.
//
// What bounds it.  That chain: D's product, its sums into H, the next D.  16 prompts of 4096 rows, 24
// heads of 128 x 64, bf16 outputs: 307 us for 1.23 GB (181 us at the copy bandwidth); one of 32768
// rows, 32 heads of 128 x 128: 398 us, about 125 of them for the segments' sums (1.1 us a chunk), 5
// for their chain, 265 for the outputs (2.3 us a chunk).  Without conversions and most products a
// chunk still takes three quarters of that, so neither tensor cores (50 to 69 % busy) nor issue slots
// (51 to 58 %) are the limit, but signals from role to role.  Tried and not faster: H in eight warps
// of 64 channels (440 against 432 us), one commit for D's and the outputs' products.
//
// Few long prompts: the rows of a request are cut into segments.  A first launch computes what
// each segment adds to a zero state, a second chains these sums, and the segments then run at
// the same time, each from its own state.
#include <algorithm>
#include <type_traits>

#include "recurrence.cuh"
#include "tc_common.cuh"

namespace tv {
namespace {

constexpr int kC = 64;        // rows per chunk
constexpr int kMaxStages = 3; // chunks of q, k, v in flight
constexpr int kWarps = 32;
constexpr int kScoreWarps = 3;  // of P
constexpr int kThreadsT = kWarps * 32;
constexpr int kWaitTries = 1 << 20;  // 7800 cycles each at most: some 4 s
constexpr uint32_t kSlab = kC * 128; // 64 rows of 64 channels
constexpr int kSpan = 120;           // log2 units that L may span in a chunk
constexpr int kSorted = 64;          // requests whose lengths the plan sorts

enum { kB, kW, kE };  // Slot::factor
enum Flags { kFirst = 1, kLast = 2, kEnd = 4 };

// What the roles need to know of a chunk.
struct alignas(16) Slot {
    float factor[3][kC];  // 2^{R - L}, 2^{d - L}, 2^{L - R}
    float2 d;             // 2^d as a pair
    float r;              // 2^R
    int row, cnt, flags, head;
    long long src, dst;   // states: a (request, head), or ~index of one in the workspace
};

struct TcParams {
    PrefillArgs a;
    int seg;        // rows per segment, a multiple of kC
    int pieces;     // segments of a request of max_rows rows
    float *states;  // [B][pieces][H][dk][dv]: the state before each segment
    float2 *decays; // [B][pieces][H]
    int sorted;     // items in order of their requests' lengths (at most kSorted requests)
    int expire;     // test hook: leave the first chunk's copies out
};

template <int DK, int DV, int NP, bool OUT>
struct Lay {
    static constexpr bool kScaleV = DV < DK;
    static constexpr int kX = kScaleV ? DV : DK;  // width of the scaled factor
    // Warps by role.  A warp reaches the lanes 32 (warp % 4) .. of tensor memory and issues from
    // scheduler warp % 4: with dv = 64 nothing lies in the upper lanes, and what does not touch
    // tensor memory goes to the warps that would be H's and the outputs' there.
    //   always   2: D's product   31: the outputs' products   24, 25, 1: P
    //   dv 128   0: plan, copies  4-19: H  20-23: outputs  3, 26-30: K~  (dk 64: 3, 26-28, 30 copies)
    //   dv 64    22: plan  23: copies  quadrants 0, 1 of 4-19: H, 2, 3: V~ or K~  20, 21: outputs
    // Without outputs 3 and 20-30 scale and 31 copies where dv is 128.
    static constexpr int kScaleWarps = DV == 64 ? 8 : !OUT ? 12 : kX == 64 ? 4 : 6;
    static constexpr int kPlanWarp = DV == 64 ? 22 : 0;
    static constexpr int kCopyWarp = DV == 64 ? 23 : !OUT ? 31 : kX == 64 ? 30 : -1;  // -1: the plan's
    __device__ static int scale_index(int warp) {  // -1: not one of them
        if (DV == 64)
            return warp >= 4 && warp < 20 && warp % 4 >= 2 ? (warp - 4) / 4 * 2 + warp % 4 - 2 : -1;
        const int from = OUT ? 26 : 20;
        return warp == 3 ? 0 : warp >= from && warp < from - 1 + kScaleWarps ? warp - from + 1 : -1;
    }
    static constexpr uint32_t kQ = 0, kK = OUT ? DK * 128 : 0, kV = kK + DK * 128,
                              kStage = kV + DV * 128;
    static constexpr int kStages = OUT && DK == 128 && DV == 128 ? 2 : kMaxStages;
    // Buffers of D (no more than stages, see the barriers' rule)
    static constexpr int kDBufs = !OUT ? 3 : DK == 64 ? 2 : 1;
    static constexpr int kAhead = 4;  // chunks that the plan may be ahead of the copies
    static constexpr int kSlots = kStages + kAhead + std::max(2, kDBufs);  // see the plan's wait
    static constexpr int kXBufs = 2;
    static constexpr uint32_t kXt = kStages * kStage, kXPart = kX * 128, kXBuf = 3 * kXPart;
    static constexpr uint32_t kP = kXt + kXBufs * kXBuf, kPPart = kC * 128;
    static constexpr uint32_t kPBuf = NP * kPPart;
    static constexpr uint32_t kOther = kSlots * (uint32_t)sizeof(Slot) + kSorted + 1024;
    static constexpr int kPBufs = kP + 2 * kPBuf + kOther <= tcc::kSmemLimit - 512 ? 2 : 1;
    static constexpr uint32_t kSlot0 = kP + (OUT ? kPBufs * kPBuf : 0), kBytes = kSlot0 + kOther;
    // tensor memory columns
    static constexpr uint32_t tD = 0, tH = kDBufs * DK, tO = tH + NP * DK / 2, tS = tO + 2 * kC, kCols = 512;
    static constexpr int kSBufs = tS + 2 * kC <= kCols ? 2 : 1;
    static_assert(OUT ? tS + kSBufs * kC <= kCols : kDBufs * DK <= kCols, "tensor memory");
    static_assert(kDBufs <= kStages, "see the barriers' rule");
    static_assert(kBytes <= tcc::kSmemLimit - 512, "shared memory");
};

// (bits of floats, as tensor memory and shared memory hold them)
using tv::halves;
using tv::two;
__device__ __forceinline__ Two two(uint32_t lo, uint32_t hi) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ void halves(Two x, uint32_t &lo, uint32_t &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(x));
}

// A pair as NP packed pairs of bf16 parts: upper bits cut off, the last part rounded.
template <int NP>
__device__ __forceinline__ void split_pair(Two x, uint32_t (&part)[NP]) {
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

constexpr int kFrac = 40;  // bits below a log2 unit: 64 rows of 4096 units take 18 above

// g log2 e in 2^-40, by a whole product of the mantissa (|g| at most 2839: 4096 log2 units); 0 for
// a NaN.  Bits below are cut off, in the same direction for all rows of one slow decay: 65536 rows
// of them are 4e-8 of a weight (in units of 2^-32 it would be 1e-5).
__device__ __forceinline__ long long log2_fixed(float g) {
    const float x = fminf(fabsf(g), 2839.f);
    const uint32_t bits = __float_as_uint(x), m = (bits & 0x7FFFFFu) | 0x800000u;
    // x = m 2^(e - 150), log2 e = 3098164009 2^-31: the product's unit is 2^(e - 181)
    const uint32_t shift = 181u - kFrac - (bits >> 23);  // 3 at least (and subnormals end as zero)
    const unsigned long long p = (unsigned long long)m * 3098164009u;  // below 2^56
    const unsigned long long y = shift < 64 ? p >> shift : 0;
    const long long z = g < 0.f ? -(long long)y : (long long)y;
    return g == g ? z : 0;
}

// 2^(x 2^-40) as a pair: a whole power and the rest of at most half a unit, rounded to 2^-32.
// (The plan's instructions are on the way from chunk to chunk: 16 prompts of 128 x 64 took 330 us
// with rows rounded and a rest of 40 bits, 304 so.)
__device__ __forceinline__ rec::Pair exp2_fixed(long long x) {
    x += 1LL << (kFrac - 33);
    const int low = (int)(x >> (kFrac - 32));
    const int n = (int)(x >> kFrac) + ((uint32_t)low >> 31);
    return rec::exp2_pair((float)n, (float)low * 2.3283064365386963e-10f);
}
// The same as one float, by the hardware's exponential (2^-22) of the rest.
__device__ __forceinline__ float exp2_single(long long x) {
    const int low = (int)(x >> (kFrac - 32));  // from a half on it counts as negative
    const int n = (int)(x >> kFrac) + ((uint32_t)low >> 31);
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"((float)low * 2.3283064365386963e-10f));
    return e * __int_as_float((max(min(n, 128), -127) + 127) << 23);
}

// 2^x and 2^-x of rows within a chunk's span, by one split of x.
__device__ __forceinline__ void exp2_both(long long x, float &up, float &down) {
    const int low = (int)(x >> (kFrac - 32));
    const int n = max(min((int)(x >> kFrac) + (int)((uint32_t)low >> 31), 127), -127);
    const float f = (float)low * 2.3283064365386963e-10f;
    float e0, e1;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(f));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(-f));
    up = e0 * __int_as_float((127 + n) << 23);
    down = e1 * __int_as_float((127 - n) << 23);
}

// Segments of a request of n rows.
__device__ __forceinline__ int pieces_of(int n, int seg) {
    return max(1, (int)(((long long)n + seg - 1) / seg));
}

// A CTA's walk over its chunks.  An item is a segment of a request and head; a CTA begins with
// the item of its block index and then takes over items of CTAs that have not been launched, so
// that long and short ones even out: the longest requests first, where there are more items than
// SMs (12 requests of up to 3000 rows, 32 heads: 240 us in the order given).
struct Walk {
    int item;              // (place * pieces + segment) * H + head, without the last segments if !OUT
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
    using L = Lay<DK, DV, NP, OUT>;
    constexpr int kStages = L::kStages, kSlots = L::kSlots;
    constexpr int kQuads = DV / 32;           // quadrants of lanes that hold something
    constexpr int kChan = DK / 4;             // channels of a lane of the H warps
    extern __shared__ uint8_t s_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ __align__(8) uint64_t s_gate[kSlots], s_full[kStages], s_s_full[2], s_p_full[2],
        s_x_full[2], s_h_full, s_h_free, s_d_full[kStages], s_d_free[L::kDBufs], s_o_full[kStages], s_o_free[2],
        s_copied[L::kAhead], s_drain[2], s_asked;
    __shared__ __align__(16) uint64_t s_answer[2];
    const PrefillArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid % 32;
    const int warp = __shfl_sync(0xffffffffu, tid / 32, 0);  // (known to be the whole warp's)
    uint8_t *s_base = s_raw + ((1024 - (ptx::smem_addr(s_raw) & 1023)) & 1023);
    const uint32_t base = ptx::smem_addr(s_base);
    Slot *slots = reinterpret_cast<Slot *>(s_base + L::kSlot0);
    uint8_t *s_order = reinterpret_cast<uint8_t *>(slots + kSlots);  // requests by length: the plan's

    const auto bar = [](const uint64_t &b) { return ptx::smem_addr(&b); };
    if (tid == 0) {
        s_abort = 0;
        for (int i = 0; i < kSlots; ++i) ptx::mbar_init(bar(s_gate[i]), 1);
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(bar(s_full[i]), 1);
            ptx::mbar_init(bar(s_d_full[i]), 1);
            ptx::mbar_init(bar(s_o_full[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(s_s_full[i]), 1);
            ptx::mbar_init(bar(s_p_full[i]), kScoreWarps);
            ptx::mbar_init(bar(s_x_full[i]), L::kScaleWarps);
            ptx::mbar_init(bar(s_o_free[i]), kQuads);
        }
        ptx::mbar_init(bar(s_h_full), 4 * kQuads);
        ptx::mbar_init(bar(s_h_free), 1);
        for (int i = 0; i < L::kDBufs; ++i) ptx::mbar_init(bar(s_d_free[i]), 4 * kQuads);
        for (int i = 0; i < L::kAhead; ++i) ptx::mbar_init(bar(s_copied[i]), 1);
        ptx::mbar_init(bar(s_drain[0]), 1);
        ptx::mbar_init(bar(s_drain[1]), 1);
        ptx::mbar_init(bar(s_asked), 1);
        ptx::fence_mbar_init();
        if (OUT) ptx::prefetch_tensormap(&map_q);
        ptx::prefetch_tensormap(&map_k);
        ptx::prefetch_tensormap(&map_v);
    }
    if (warp == 2) {
        ptx::tmem_alloc(ptx::smem_addr(&s_tmem), L::kCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
    pdl_wait();
    pdl_launch_next();

    // A wait that expires raises the CTA's flag and its warp leaves; the others' expire in turn.
    // (The whole wait is one short loop, and what a warp does next is a vote: the compiler then
    // knows that warps stay whole, and keeps the products' operands in uniform registers.)
    const int tries = p.expire ? kWaitTries / 64 : kWaitTries;
    const auto wait = [&](const uint64_t &b, uint32_t parity) {
        const bool ok = __all_sync(0xffffffffu, ptx::mbar_wait_tries(bar(b), parity, tries));
        if (!ok) *(volatile int *)&s_abort = 1;
        return ok;
    };
    const auto arrive = [&](const uint64_t &b) {  // once per warp, after all of its lanes
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(b));
    };
    // No barrier runs a phase ahead of those who wait for it: whoever completes chunk n's phase
    // needs something of every waiter's for chunk n - 1 (or n - 2, where there are two buffers and
    // barriers) first.
    // A role's walk over the chunks: number, slot, stage and the parities of their barriers.
    struct Turn {
        int n = 0, slot = 0, stage = 0;
        uint32_t slot_ph = 0, stage_ph = 0;
        __device__ void next() {
            ++n;
            if (++slot == kSlots) {
                slot = 0;
                slot_ph ^= 1;
            }
            if (++stage == kStages) {
                stage = 0;
                stage_ph ^= 1;
            }
        }
    };
    // the chunk's flags once its decays are there; kEnd if there is none
    const auto gate = [&](const Turn &t) {
        if (!wait(s_gate[t.slot], t.slot_ph)) return (int)kEnd;
        return (int)__reduce_or_sync(0xffffffffu, (uint32_t)slots[t.slot].flags);
    };

    // The rows of a chunk on their way to a stage, by one lane; whole at t's phase of s_full.
    const auto copy = [&](const Turn &t, int head, int row) {
        if (lane == 0) {
            const uint32_t at = base + t.stage * L::kStage, full = bar(s_full[t.stage]);
            ptx::mbar_arrive_expect_tx(full, OUT ? L::kStage : L::kStage - L::kK);
            ptx::tma_load_4d(at + L::kK, &map_k, 0, head, row, 0, full);
            ptx::tma_load_4d(at + L::kV, &map_v, 0, head, row, 0, full);
            if (OUT) ptx::tma_load_4d(at + L::kQ, &map_q, 0, head, row, 0, full);
        }
        __syncwarp();
    };
    // The products of the chunk that had t's stage are done.
    const auto stage_free = [&](const Turn &t) {
        return t.n < kStages || (wait(s_d_full[t.stage], t.stage_ph ^ 1) &&
                                 (!OUT || wait(s_o_full[t.stage], t.stage_ph ^ 1)));
    };
    // Copies that nobody waited for (after a timeout) may not land later.
    const auto copies_end = [&](int issued) {
        if (*(volatile int *)&s_abort)
            for (int i = max(0, issued - kStages); i < issued; ++i)
                ptx::mbar_wait_tries(bar(s_full[i % kStages]), (i / kStages) & 1, 1 << 14);
    };

    const int scale = L::scale_index(warp);
    if (warp == L::kPlanWarp) {
        // ---- plan, decays and copies
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
                const int slot = w.item / a.H, place = slot / per, i = slot - place * per;
                const int b = p.sorted ? s_order[place] : place;
                int off, n;
                if (!request_range(a.offsets, b, a.R, a.max_rows, off, n)) {
                    if (lane == 0) report(a.status, TV_ERR_TREE);
                    continue;
                }
                const int pieces = pieces_of(n, p.seg);
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
        if (p.sorted) {
            const auto rows = [&](int b) {
                int off, n = 0;
                return b < a.B && request_range(a.offsets, b, a.R, a.max_rows, off, n) ? n : 0;
            };
#pragma unroll 1
            for (int b0 = 0; b0 < a.B; b0 += 32) {
                const int b = b0 + lane, n = rows(b);
                int place = 0;
#pragma unroll 1
                for (int j0 = 0; j0 < a.B; j0 += 32) {
                    const int m = rows(j0 + lane);
#pragma unroll 1
                    for (int j = j0; j < min(a.B, j0 + 32); ++j) {
                        const int x = __shfl_sync(0xffffffffu, m, j - j0);
                        place += x > n || (x == n && j < b);
                    }
                }
                if (b < a.B) s_order[place] = b;
            }
            __syncwarp();
        }
        next_item(true);
        // decays of the chunk at w, and of the 64 rows that begin at `ahead`, on their way from memory
        // for a whole turn
        float g0 = 0.f, g1 = 0.f, next0 = 0.f, next1 = 0.f;
        int ahead = -1;
        const auto load = [&](int row, float &x0, float &x1) {
            const int t = row + 2 * lane;
            const float *g = a.g + w.head + (size_t)t * a.g_stride;
            x0 = !w.done && t < w.end ? g[0] : 0.f;
            x1 = !w.done && t + 1 < w.end ? g[a.g_stride] : 0.f;
        };
        const auto fetch = [&]() {
            g0 = next0;
            g1 = next1;
            if (w.first || w.row != ahead) load(w.row, g0, g1);
            ahead = w.row + kC;
            load(ahead, next0, next1);
        };
        fetch();
        long long total = 0;  // log2 of the item's decay so far
        bool total_nan = false;
        int issued = 0;
        for (Turn t;; t.next()) {
            Slot *s = slots + t.slot;
            if (w.done) {
                if (L::kCopyWarp >= 0 && t.n >= L::kAhead &&
                    !wait(s_copied[t.n % L::kAhead], (t.n / L::kAhead & 1) ^ 1))
                    break;
                if (lane == 0) s->flags = kEnd;
                arrive(s_gate[t.slot]);
                break;
            }
            if (p.expire) {
                wait(s_asked, (w.asked - 1) & 1);
                break;
            }
            const int row = w.row, head = w.head;
            int cnt = min(kC, w.end - row);
            const bool nan0 = g0 != g0, nan1 = g1 != g1;
            const long long y0 = log2_fixed(g0), y1 = log2_fixed(g1);
            long long sum = y0 + y1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            const long long l0 = sum - y1, l1 = sum;
            long long end = __shfl_sync(0xffffffffu, sum, 31);
            const int h0 = (int)(l0 >> kFrac), h1 = (int)(l1 >> kFrac);
            int lo = __reduce_min_sync(0xffffffffu, min(h0, h1));
            int hi = __reduce_max_sync(0xffffffffu, max(h0, h1));
            if (hi - lo > kSpan) {
                // the first row whose L is too far from one before it ends the chunk (rare: running
                // extremes row by row)
                lo = hi = __shfl_sync(0xffffffffu, h0, 0);
                for (int r = 1; r < cnt; ++r) {
                    const int h = __shfl_sync(0xffffffffu, r & 1 ? h1 : h0, r / 2);
                    if (max(hi, h) - min(lo, h) > kSpan) {
                        cnt = r;
                        const long long e0 = __shfl_sync(0xffffffffu, l0, (r - 1) / 2);
                        const long long e1 = __shfl_sync(0xffffffffu, l1, (r - 1) / 2);
                        end = (r - 1) & 1 ? e1 : e0;
                        break;
                    }
                    lo = min(lo, h);
                    hi = max(hi, h);
                }
            }
            const long long mid = (long long)((lo + hi) / 2) * (1LL << kFrac);
            const bool first = w.first, last = row + cnt >= w.end;
            const long long unit_of = w.unit, ws = w.ws;
            const bool cut = w.pieces > 1, final_piece = w.piece == w.pieces - 1;
            w.first = false;
            w.row += cnt;
            if (last) next_item(false);
            fetch();  // the next chunk's, on its way while this one's become factors

            // The slot is free: the copies of kAhead chunks earlier found their stage free, so the
            // products of the chunk that had that stage are done.  These waited for the outputs of
            // two chunks earlier to be read, and for H's sums of kDBufs chunks earlier.
            if (L::kCopyWarp >= 0 && t.n >= L::kAhead &&
                !wait(s_copied[t.n % L::kAhead], (t.n / L::kAhead & 1) ^ 1))
                break;

            // from the first NaN on, everything of this request and head is one
            const uint32_t within = 2 * lane < cnt ? 1u : 0u;
            const uint32_t bad0 = __ballot_sync(0xffffffffu, nan0 && within),
                           bad1 = __ballot_sync(0xffffffffu, nan1 && 2 * lane + 1 < cnt);
            const bool any = (bad0 | bad1) != 0;
            const float nanf = __int_as_float(0x7fffffff);
            float2 ev = make_float2(0.f, 0.f), bv = ev;
            if (OUT) {
                exp2_both(l0 - mid, ev.x, bv.x);
                exp2_both(l1 - mid, ev.y, bv.y);
                *reinterpret_cast<float2 *>(s->factor[kB] + 2 * lane) = bv;
            }
            *reinterpret_cast<float2 *>(s->factor[kW] + 2 * lane) =
                make_float2(exp2_single(end - l0), exp2_single(end - l1));
            if (OUT) {
                if (any) {
                    const uint32_t upto = 0xffffffffu >> (31 - lane);
                    if ((bad0 & upto) || (bad1 & (upto >> 1))) ev.x = nanf;
                    if ((bad0 | bad1) & upto) ev.y = nanf;
                }
                *reinterpret_cast<float2 *>(s->factor[kE] + 2 * lane) = ev;
            }
            if (first) {
                total = 0;
                total_nan = false;
            }
            // (2^20 units either way are as good as any more, and many rows of 4096 may not wrap around)
            total = max(min(total + end, 1LL << 60), -(1LL << 60));
            total_nan |= any;
            const rec::Pair d = exp2_fixed(end);
            const float r = exp2_single(mid);
            if (lane == 0) {
                s->d = any ? make_float2(nanf, nanf) : make_float2(d.hi, d.lo);
                s->r = r;
                s->row = row;
                s->cnt = cnt;
                s->head = head;
                s->flags = (first ? kFirst : 0) | (last ? kLast : 0);
                if (OUT) {
                    s->src = cut ? ~ws : unit_of;
                    s->dst = final_piece ? unit_of : -1;
                } else {
                    s->src = -1;
                    s->dst = ~(ws + a.H);  // where the next segment begins
                    if (last) {
                        const rec::Pair d = exp2_fixed(total);
                        p.decays[ws] = total_nan ? make_float2(nanf, nanf) : make_float2(d.hi, d.lo);
                    }
                }
            }
            arrive(s_gate[t.slot]);
            // (With a warp for the copies the plan goes by its word alone: chunk n's products may be
            // done, and their barriers a phase on, before the plan has looked at them.)
            if (L::kCopyWarp < 0) {
                if (!stage_free(t)) break;
                copy(t, head, row);
                issued = t.n + 1;
            }
        }
        copies_end(issued);
    } else if (warp == L::kCopyWarp) {
        // ---- copies
        int issued = 0;
        for (Turn t;; t.next()) {
            if (gate(t) & kEnd) break;
            const int head = slots[t.slot].head, row = slots[t.slot].row;
            if (!stage_free(t)) break;
            arrive(s_copied[t.n % L::kAhead]);  // (head and row have been read too)
            copy(t, head, row);
            issued = t.n + 1;
        }
        copies_end(issued);
    } else if (warp == 2) {
        // ---- what a chunk adds to the state: D^T = V^T K~ (or V~^T K)
        const uint32_t lead = ptx::elect_one();
        for (Turn t;; t.next()) {
            if (gate(t) & kEnd) break;
            const int xb = t.n % L::kXBufs, db = t.n % L::kDBufs;
            if (!wait(s_full[t.stage], t.stage_ph)) break;
            if (t.n >= L::kDBufs && !wait(s_d_free[db], (t.n / L::kDBufs & 1) ^ 1)) break;
            if (!wait(s_x_full[xb], (t.n / L::kXBufs) & 1)) break;
            ptx::tc_fence_after_sync();
            // descriptors move by their address field, in units of 16 bytes
            const uint32_t st = base + t.stage * L::kStage;
            const uint64_t raw =
                ptx::desc_mnmajor_sw128(st + (L::kScaleV ? L::kK : L::kV), kSlab, 1024);
            const uint64_t scaled =
                ptx::desc_mnmajor_sw128(base + L::kXt + xb * L::kXBuf, kSlab, 1024);
#pragma unroll
            for (int part = 2; part >= 0; --part)
#pragma unroll
                for (int kk = 0; kk < kC / 16; ++kk) {
                    const uint64_t x = scaled + part * (L::kXPart / 16) + kk * 128;
                    const uint64_t y = raw + kk * 128;
                    ptx::mma_bf16_lead(tmem + L::tD + db * DK, L::kScaleV ? x : y, L::kScaleV ? y : x,
                                       ptx::idesc_bf16_f32_abmn(128, DK), part < 2 || kk > 0, lead);
                }
            ptx::mma_commit_lead(bar(s_d_full[t.stage]), lead);
        }
        ptx::mma_commit_lead(bar(s_drain[0]), lead);
        __syncwarp();
        ptx::mbar_wait_tries(bar(s_drain[0]), 0, 1 << 18);
    } else if (OUT && warp == 31) {
        // ---- the outputs' products: S, H^T Q^T and V^T P^T
        const uint32_t lead = ptx::elect_one();
        const auto scores = [&](const Turn &t) {
            // 128 lanes take the 64 rows behind the tile along; nobody reads their results
            const uint32_t st = base + t.stage * L::kStage, buf = t.n % L::kSBufs;
            const uint64_t q = ptx::desc_kmajor_sw128(st + L::kQ, 1024),
                           k = ptx::desc_kmajor_sw128(st + L::kK, 1024);
#pragma unroll
            for (int kk = 0; kk < DK / 16; ++kk) {
                const uint32_t o = (kk / 4 * kSlab + kk % 4 * 32) / 16;
                ptx::mma_bf16_lead(tmem + L::tS + buf * kC, q + o, k + o,
                                   ptx::idesc_bf16_f32(128, kC), kk > 0, lead);
            }
            ptx::mma_commit_lead(bar(s_s_full[buf]), lead);
        };
        Turn t;
        bool ok = !(gate(t) & kEnd);
        if (ok) {
            ok = wait(s_full[0], 0);
            ptx::tc_fence_after_sync();
            if (ok) scores(t);
        }
        while (ok) {
            const int n = t.n, ob = n & 1;
            const uint32_t ph = n & 1, st = base + t.stage * L::kStage;
            const uint32_t o = tmem + L::tO + ob * kC;
            if (!__all_sync(0xffffffffu,
                            ptx::mbar_test_wait(bar(s_h_full), ph) &&
                                (n < 2 || ptx::mbar_test_wait(bar(s_o_free[ob]), ((n >> 1) & 1) ^ 1)))) {
                if (n >= 2 && !(ok = wait(s_o_free[ob], ((n >> 1) & 1) ^ 1))) break;
                if (!(ok = wait(s_h_full, ph))) break;
            }
            ptx::tc_fence_after_sync();
            const uint64_t qd = ptx::desc_kmajor_sw128(st + L::kQ, 1024);
#pragma unroll
            for (int part = NP - 1; part >= 0; --part)
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk)
                    ptx::mma_bf16_ts_lead(o, tmem + L::tH + part * (DK / 2) + kk * 8,
                                          qd + (kk / 4 * kSlab + kk % 4 * 32) / 16,
                                          ptx::idesc_bf16_f32(128, kC), part < NP - 1 || kk > 0,
                                          lead);
            ptx::mma_commit_lead(bar(s_h_free), lead);
            Turn u = t;
            u.next();
            // the next chunk's scores ahead of this one's weights, if it is there and they have
            // a buffer of their own
            bool scored = false;
            int next = -1;  // its flags, once they are known
            if (__all_sync(0xffffffffu, ptx::mbar_test_wait(bar(s_gate[u.slot]), u.slot_ph))) {
                next = (int)__reduce_or_sync(0xffffffffu, (uint32_t)slots[u.slot].flags);
                if (L::kSBufs == 2 && !(next & kEnd) &&
                    __all_sync(0xffffffffu, ptx::mbar_test_wait(bar(s_full[u.stage]), u.stage_ph))) {
                    ptx::tc_fence_after_sync();
                    scores(u);
                    scored = true;
                }
            }
            const int pb = n % L::kPBufs;
            if (!(ok = wait(s_p_full[pb], (n / L::kPBufs) & 1))) break;
            ptx::tc_fence_after_sync();
            const uint64_t vd = ptx::desc_mnmajor_sw128(st + L::kV, kSlab, 1024);
            const uint64_t pd = ptx::desc_kmajor_sw128(base + L::kP + pb * L::kPBuf, 1024);
#pragma unroll
            for (int part = NP - 1; part >= 0; --part)
#pragma unroll
                for (int kk = 0; kk < kC / 16; ++kk)
                    ptx::mma_bf16_lead(o, vd + kk * 128, pd + part * (L::kPPart / 16) + kk * 2,
                                       ptx::idesc_bf16_f32_amn(128, kC), 1, lead);
            ptx::mma_commit_lead(bar(s_o_full[t.stage]), lead);
            t = u;
            if (next < 0) next = gate(t);
            if (next & kEnd) break;
            if (!scored) {
                // (P of the chunk before has been written, so its scores have been read)
                if (!(ok = wait(s_full[t.stage], t.stage_ph))) break;
                ptx::tc_fence_after_sync();
                scores(t);
            }
        }
        ptx::mma_commit_lead(bar(s_drain[1]), lead);
        __syncwarp();
        ptx::mbar_wait_tries(bar(s_drain[1]), 0, 1 << 18);
    } else if (scale >= 0) {
        // ---- K~ or V~: rows times 2^{d - L}, in three parts, laid out as the rows are.  A few
        // threads to a row; a quarter warp's eight rows keep their 16-byte pieces on different
        // banks.
        const int i0 = scale * 32 + lane, r = i0 % kC, sub = i0 / kC;
        constexpr int kSubs = L::kScaleWarps / 2;
        const uint32_t line = r * 128, swz = (r & 7) * 16;
        for (Turn t;; t.next()) {
            // (what the chunk needs, tested together: a test that finds its phase complete takes
            // a few hundred cycles when shared memory is busy)
            const int was = t.n - L::kXBufs;  // the chunk whose product read the buffer last
            const bool all = __all_sync(
                0xffffffffu,
                ptx::mbar_test_wait(bar(s_gate[t.slot]), t.slot_ph) &
                    ptx::mbar_test_wait(bar(s_full[t.stage]), t.stage_ph) &
                    (was < 0 ||
                     ptx::mbar_test_wait(bar(s_d_full[was % kStages]), (was / kStages) & 1)));
            if (!all && !wait(s_gate[t.slot], t.slot_ph)) break;
            const Slot *s = slots + t.slot;
            if (__any_sync(0xffffffffu, s->flags & kEnd)) break;
            const int cnt = s->cnt;
            const bool live = r < cnt;
            const float w = live ? s->factor[kW][r] : 0.f;  // (past the chunk it may be infinite)
            const Two w2 = two(w, w);
            const int xb = t.n % L::kXBufs;
            if (!all && (!wait(s_full[t.stage], t.stage_ph) ||
                         (was >= 0 && !wait(s_d_full[was % kStages], (was / kStages) & 1))))
                break;
            uint8_t *st = s_base + t.stage * L::kStage;
            if (cnt < kC) {  // rows past the chunk may hold anything: the products take zeros
                const uint4 zero = make_uint4(0, 0, 0, 0);
                if (!live) {
                    for (int c = sub; c < DV / 8; c += kSubs)
                        *reinterpret_cast<uint4 *>(st + L::kV + c / 8 * kSlab + line + c % 8 * 16) = zero;
                    for (int c = sub; c < DK / 8; c += kSubs)
                        *reinterpret_cast<uint4 *>(st + L::kK + c / 8 * kSlab + line + c % 8 * 16) = zero;
                }
            }
            const uint8_t *from = st + (L::kScaleV ? L::kV : L::kK);
            uint8_t *to = s_base + L::kXt + xb * L::kXBuf;
#pragma unroll 2
            for (int c = sub; c < L::kX / 8; c += kSubs) {
                const uint32_t at = c / 8 * kSlab + line + ((c % 8 * 16) ^ swz);
                uint4 x = make_uint4(0, 0, 0, 0);
                if (live) x = *reinterpret_cast<const uint4 *>(from + at);
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
                    *reinterpret_cast<uint4 *>(to + j * L::kXPart + at) =
                        make_uint4(out[j][0], out[j][1], out[j][2], out[j][3]);
            }
            ptx::fence_proxy_async_smem();
            arrive(s_x_full[xb]);
        }
    } else if (warp >= 4 && warp < 20) {
        // ---- H: lane = column of the state, kChan of its channels in registers
        const int quad = warp % 4, c0 = (warp - 4) / 4 * kChan, col = quad * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)quad << 21);  // lane quad * 32
        if (quad < kQuads) {
            Two h[kChan / 2];
            Turn t;
            int flags = gate(t);
            while (!(flags & kEnd)) {
                const Slot *s = slots + t.slot;
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
                    const Two r2 = two(s->r, s->r);
                    bool ok = true;
#pragma unroll
                    for (int i0 = 0; i0 < kChan / 2; i0 += 8) {
                        uint32_t part[NP][8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            uint32_t x[NP];
                            split_pair<NP>(mul2(h[i0 + i], r2), x);
#pragma unroll
                            for (int j = 0; j < NP; ++j) part[j][i] = x[j];
                        }
                        if (i0 == 0 && t.n > 0) {  // the chunk's before are read
                            if (!(ok = wait(s_h_free, (t.n & 1) ^ 1))) break;
                            ptx::tc_fence_after_sync();
                        }
#pragma unroll
                        for (int j = 0; j < NP; ++j)
                            ptx::tmem_st_x8(lanes + L::tH + j * (DK / 2) + c0 / 2 + i0, part[j]);
                    }
                    if (!ok) break;
                    ptx::tmem_wait_st();
                }
                const int db = t.n % L::kDBufs;
                const Two dx = two(s->d.x, s->d.x), dy = two(s->d.y, s->d.y);
                const long long dst = s->dst;
                if (OUT) {
                    ptx::tc_fence_before_sync();
                    arrive(s_h_full);
                }
                // (the next chunk's flags while D is on its way)
                Turn u = t;
                u.next();
                const int next = gate(u);
                if (!wait(s_d_full[t.stage], t.stage_ph)) break;
                ptx::tc_fence_after_sync();
#pragma unroll
                for (int i0 = 0; i0 < kChan; i0 += 16) {
                    uint32_t x[16];
                    ptx::tmem_ld_x16_nowait(lanes + L::tD + db * DK + c0 + i0, x);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        Two &y = h[i0 / 2 + i];
                        y = fma2(y, dx, fma2(y, dy, two(x[2 * i], x[2 * i + 1])));
                    }
                }
                ptx::tc_fence_before_sync();
                arrive(s_d_free[db]);
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
                t = u;
                flags = next;
            }
        }
    } else if (warp >= 20 && warp < 24) {
        // ---- outputs: lane = column, 64 rows.  bf16: neighbouring lanes trade halves, so that an
        // even lane stores both columns of an even row and an odd lane those of the next.
        const int quad = warp % 4, col = quad * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)quad << 21);
        if (OUT && quad < kQuads) {
            const uint32_t step = (uint32_t)a.H * DV;  // elements from row to row
            for (Turn t;; t.next()) {
                if (gate(t) & kEnd) break;
                const Slot *s = slots + t.slot;
                const int cnt = s->cnt, ob = t.n & 1;
                const size_t at = ((size_t)s->row * a.H + s->head) * DV;
                if (!wait(s_o_full[t.stage], t.stage_ph)) break;
                ptx::tc_fence_after_sync();
#pragma unroll 1
                for (int t0 = 0; t0 < kC; t0 += 16) {
                    uint32_t x[16];
                    ptx::tmem_ld_x16_nowait(lanes + L::tO + ob * kC + t0, x);
                    const float4 *e4 = reinterpret_cast<const float4 *>(s->factor[kE] + t0);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 f = e4[i];
                        const Two o01 = mul2(two(f.x, f.y), two(x[4 * i], x[4 * i + 1]));
                        const Two o23 = mul2(two(f.z, f.w), two(x[4 * i + 2], x[4 * i + 3]));
                        uint32_t o[4];
                        halves(o01, o[0], o[1]);
                        halves(o23, o[2], o[3]);
                        const int r = t0 + 4 * i;
                        if (NP == 3) {
                            float *to = static_cast<float *>(a.out) + at + col;
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                if (r + u < cnt)
                                    to[(size_t)(uint32_t)(r + u) * step] = __uint_as_float(o[u]);
                        } else {
                            const int odd = lane & 1;
                            __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(a.out) + at + (col - odd);
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const __nv_bfloat162 b = __floats2bfloat162_rn(
                                    __uint_as_float(o[2 * u]), __uint_as_float(o[2 * u + 1]));
                                const uint32_t own = *reinterpret_cast<const uint32_t *>(&b);
                                const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
                                const int rr = r + 2 * u + odd;
                                if (rr < cnt)
                                    *reinterpret_cast<uint32_t *>(to + (size_t)(uint32_t)rr * step) =
                                        __byte_perm(own, other, odd ? 0x3276 : 0x5410);
                            }
                        }
                    }
                }
                ptx::tc_fence_before_sync();
                arrive(s_o_free[ob]);
            }
        }
    } else if (warp == 24 || warp == 25 || warp == 1) {
        // ---- P: lane = row of the chunk; two blocks of 16 columns each for warp 24 (rows 0-31,
        // which reach no further), 25 and 1 (rows 32-63)
        if (OUT) {
            const int quad = warp % 4, i = quad * 32 + lane, from = warp == 1 ? 2 : 0;
            const uint32_t lanes = tmem + ((uint32_t)quad << 21);
            uint8_t *row = s_base + L::kP + i * 128;
            if (warp == 24)  // zero once and for all: columns past the rows
                for (int c = 4; c < 8; ++c)
                    for (int j = 0; j < NP * L::kPBufs; ++j)
                        *reinterpret_cast<uint4 *>(row + j * L::kPPart + ((c ^ (i & 7)) * 16)) =
                            make_uint4(0, 0, 0, 0);
            for (Turn t;; t.next()) {
                if (gate(t) & kEnd) break;
                const Slot *s = slots + t.slot;
                const int sb = t.n % L::kSBufs;
                if (!wait(s_s_full[sb], (t.n / L::kSBufs) & 1)) break;
                if (s->cnt < kC) {  // rows past the chunk: V as V^T P^T takes it (K~'s warps see to
                                    // the other product on their own)
                    const int w3 = warp == 1 ? 2 : warp - 24, rows = kC - s->cnt;
                    uint8_t *v = s_base + t.stage * L::kStage + L::kV + s->cnt * 128;
                    for (int z = w3 * 32 + lane; z < rows * (DV / 8); z += 96)
                        *reinterpret_cast<uint4 *>(v + z / (rows * 8) * kSlab + z % (rows * 8) * 16) =
                            make_uint4(0, 0, 0, 0);
                }
                const int was = t.n - L::kPBufs;  // its P has been read
                if (was >= 0 && !wait(s_o_full[was % kStages], (was / kStages) & 1)) break;
                uint8_t *mine = row + t.n % L::kPBufs * L::kPBuf;
                ptx::tc_fence_after_sync();
#pragma unroll 1
                for (int jb = from; jb < from + 2; ++jb) {
                    uint32_t x[16];
                    ptx::tmem_ld_x16_nowait(lanes + L::tS + sb * kC + jb * 16, x);
                    const float4 *b4 = reinterpret_cast<const float4 *>(s->factor[kB] + jb * 16);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t out[NP][4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float4 b = b4[2 * c + h];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int u = 8 * c + 4 * h + 2 * e, j = jb * 16 + u;
                                uint32_t y0, y1, part[NP];
                                halves(mul2(two(x[u], x[u + 1]), e ? two(b.z, b.w) : two(b.x, b.y)),
                                       y0, y1);
                                split_pair<NP>(two(j <= i ? y0 : 0u, j < i ? y1 : 0u), part);
#pragma unroll
                                for (int q = 0; q < NP; ++q) out[q][2 * h + e] = part[q];
                            }
                        }
                        uint8_t *at = mine + (((jb * 2 + c) ^ (i & 7)) * 16);
#pragma unroll
                        for (int q = 0; q < NP; ++q)
                            *reinterpret_cast<uint4 *>(at + q * L::kPPart) =
                                make_uint4(out[q][0], out[q][1], out[q][2], out[q][3]);
                    }
                }
                ptx::tc_fence_before_sync();
                ptx::fence_proxy_async_smem();
                arrive(s_p_full[t.n % L::kPBufs]);
            }
        }
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (tid == 0 && s_abort) report(a.status, TV_ERR_TIMEOUT);
    if (warp == 2) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, L::kCols);
    }
}

// The segments' states from what each adds: S_{i+1} = 2^{d_i} S_i + added_i.  Latency bounds it (a
// dependent load each: 1 us a segment), so kChain segments' sums are on their way together.
constexpr int kThreadsChain = 256;
constexpr int kChain = 8;
__global__ void __launch_bounds__(kThreadsChain) prefill_chain_kernel(TcParams p) {
    const PrefillArgs &a = p.a;
    const int unit = blockIdx.x, b = unit / a.H, h = unit % a.H;
    const size_t quads = (size_t)a.dk * a.dv / 4, at = (size_t)blockIdx.y * kThreadsChain + threadIdx.x;
    pdl_wait();
    pdl_launch_next();
    int off, n;
    if (at >= quads || !request_range(a.offsets, b, a.R, a.max_rows, off, n)) return;
    const int pieces = pieces_of(n, p.seg);
    if (pieces < 2) return;
    const size_t first = (size_t)b * p.pieces * a.H + h;
    float4 *state = reinterpret_cast<float4 *>(p.states) + first * quads + at;
    const float2 *decay = p.decays + first;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.H0) x = reinterpret_cast<const float4 *>(a.H0)[(size_t)unit * quads + at];
    *state = x;
    for (int i0 = 1; i0 < pieces; i0 += kChain) {
        float4 y[kChain];
        float2 d[kChain];
#pragma unroll
        for (int u = 0; u < kChain; ++u) {
            const size_t i = min(i0 + u, pieces - 1);
            y[u] = state[i * a.H * quads];
            d[u] = decay[(i - 1) * a.H];
        }
#pragma unroll
        for (int u = 0; u < kChain; ++u) {
            if (i0 + u >= pieces) break;
            x.x = fmaf(x.x, d[u].x, fmaf(x.x, d[u].y, y[u].x));
            x.y = fmaf(x.y, d[u].x, fmaf(x.y, d[u].y, y[u].y));
            x.z = fmaf(x.z, d[u].x, fmaf(x.z, d[u].y, y[u].z));
            x.w = fmaf(x.w, d[u].x, fmaf(x.w, d[u].y, y[u].w));
            state[(size_t)(i0 + u) * a.H * quads] = x;
        }
    }
}

// ---------------------------------------------------------------- host side

// Chunks of the longest request that there can be.
long long most_chunks(const PrefillArgs &a) {
    return std::max(1LL, (std::min(a.max_rows, a.R) + kC - 1LL) / kC);
}

// Pieces that a request of that length is cut into: what makes the longest SM's work least,
// counted in chunks.  A segment costs a few chunks to start, and its first launch 0.6 of what a
// chunk costs (with 0.5, which is what full SMs take, few and long segments look too cheap).
// One prompt of 32768 rows and 32 heads of 128 x 128, at an earlier step: 466 us in 4 pieces, 433
// in 9 (taken), 432 in 14, 463 in 28.  Two of 16384, bf16 outputs, in 7 pieces (taken) and in 2 (by
// 0.5): 412 and 456 us, 128 x 64 324 and 364, 64 x 128 330 and 372, 64 x 64 294 and 344.  64 heads of
// 4096 rows uncut (taken) and in 2: 144 and 138, 105 and 114, 105 and 113, 98 and 104.
int best_pieces(const PrefillArgs &a) {
    const long long units = (long long)a.B * a.H, sms = device_sms(), chunks = most_chunks(a);
    if (units > 8 * sms) return 1;
    const auto waves = [&](long long items) { return (double)((items + sms - 1) / sms); };
    int best = 1;
    double least = waves(units) * (chunks + 4.0);
    for (int s = 2; s <= 64 && s <= chunks; ++s) {
        const double per = (double)((chunks + s - 1) / s);
        const double cost =
            waves(units * s) * (per + 4.0) + waves(units * (s - 1)) * (0.6 * per + 4.0) + 8.0;
        if (cost < 0.95 * least) {
            least = cost;
            best = s;
        }
    }
    return best;
}

int segment_rows(const PrefillArgs &a, int pieces) {
    return (int)std::min<long long>((most_chunks(a) + pieces - 1) / pieces * kC, 0x7fffffc0);
}

size_t cut_bytes(const PrefillArgs &a, int pieces) {
    const size_t items = (size_t)a.B * pieces * a.H;
    return items * a.dk * a.dv * 4 + (items * 8 + 15) / 16 * 16;
}

// Boxes of 64 rows of one head, in slabs of 64 channels (the last dimension, so that a box is a
// slab after the other).
bool rows_map(CUtensorMap *m, const void *base, int width, int H, int R, int64_t stride) {
    const cuuint64_t dims[4] = {64, (cuuint64_t)H, (cuuint64_t)R, (cuuint64_t)width / 64};
    const cuuint64_t strides[3] = {(cuuint64_t)width * 2, (cuuint64_t)stride * 2, 128};
    const cuuint32_t box[4] = {64, 1, kC, (cuuint32_t)width / 64}, one[4] = {1, 1, 1, 1};
    const auto encode = tcc::encode_fn();
    return encode && encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims,
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
                      Lay<DK, DV, NP, OUT>::kBytes, s, m[0], m[1], m[2], p);
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
    // (a microsecond or two of every CTA's start, lost on short requests and on equal ones)
    p.sorted = a.B <= kSorted && (long long)a.B * a.H > device_sms() && most_chunks(a) >= 8 &&
               a.R < (long long)a.B * a.max_rows;
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
           a.v_stride < most && (int64_t)a.H * a.dv < 0x7fffffff;
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
