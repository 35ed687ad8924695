// kpa_paged_prefill.cu -- attention of chunks of new tokens over a paged factor cache on the
// tcgen05 tensor cores, for d1 = 8 (d2 = 16 at R = 2 or 4, d2 = 8 at R = 2) and d1 =
// h2 = 1, TPA's split (d2 = 64 at R = 1 or 2, d2 = 128 at R = 2); every other split runs on the mma.sync
// kernel.
//
// The arrangement is the contiguous cache's prefill: one CTA takes 256 query rows of one
// (sequence, head) as two 128-row halves that share every rebuilt 128-slot K/V tile and take
// turns on the tensor pipe; a producer warp per plane streams factor slices, eight warps
// rebuild K and V^T as fp16 in the 128-byte-swizzled layouts tcgen05.mma reads, one thread
// issues S_h = Q_h K^T and O_h += P_h V, and eight softmax warps (a row per thread) turn S_h
// into P_h in tensor memory (S0 | S1 | O0 | O1, 128 columns each).  What differs:
//   - rows come flattened, each CTA finds its sequence by a scan of the row offsets;
//   - the tiles are those the CTA's rows see: the sinks' and the windows', or one of n_split
//     equal runs of them when there are few CTAs, whose partials a second kernel joins;
//   - a tile's 16-slot groups come through the page table as 16-byte asynchronous copies;
//     groups that no row sees are skipped, rebuilt slots that no row sees are zeros;
//   - a CTA with at most 128 rows has both halves work on them, on tiles in turns, each with
//     its own maxima, sums and output, joined at the end: a tile then costs its rebuild and not
//     the chain of a half's products and softmax (9 x 128 rows over 4096 slots, 4 x 4 heads of
//     8 x 16, R = 2: 90 -> 71 us);
//   - with d1 = 1 a head's slice of a slot (R (1 + d2) values) is larger than its key, so a
//     tile is staged and rebuilt in units of 4096 / d_h slots, by four warps per plane.  The
//     slice's B rows (contiguous in a group, as h2 = 1) come as one bulk copy per group: a warp
//     issues its lanes' copies one after the other, and 16 of them took 1600 clocks, longer than
//     the unit's rebuild (9 x 128 rows, 16 heads of 128, R = 2: 150 -> 100 us);
//   - an e4m3 token's two scales multiply into its factors before K and V are rounded once to
//     fp16: in fp32, or at R = 2 in fp16, where factors and products are exact.
// Bound by each half's chain of S, softmax and P V at d1 = 8 (8 x 2048 causal tokens of 4 x 4 heads
// of 8 x 16 in 255 us, 539 TFLOP/s, the tensor pipe 27 % busy), by the rebuild at d1 = 1 and in
// short row tiles.
#include <cstring>
#include <type_traits>

#include "kpa_f32x2.cuh"
#include "kpa_paged.cuh"
#include "kpa_prefill_tc.cuh"

namespace kpa {
namespace {

using namespace paged;
using namespace prefill_tc;
using f32x2::exp2_poly2;
using f32x2::fadd2;
using f32x2::ffma2;
using f32x2::fmul2;
using f32x2::fsub2;
using f32x2::unpack_bf16x2;

constexpr int HQ = 128;                       // query rows per half
constexpr int TK = 128;                       // slots per tile
constexpr int kSoftmaxWarps = 8, kRebuildWarps = 8;
constexpr int kRebuildWarp0 = kSoftmaxWarps;
constexpr int kMmaWarp = kSoftmaxWarps + kRebuildWarps;
constexpr int kProducerWarp = kMmaWarp + 1;                   // keys; the next warp, values
constexpr int kThreads = (kProducerWarp + 2) * 32;            // 608
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.f;           // the running maximum moves when it grew past 2^8

struct PrefillArgsP {
    PagedAttnArgs p;
    Pool pool;
    int h1, h2;
    unsigned long long wait_limit_ns;
};

template <int D1_, int D2_, int R_, bool E4M3_>
struct Cfg {
    static constexpr int D1 = D1_, D2 = D2_, R = R_, DH = D1 * D2, HB = D2 / 8;
    static constexpr bool E4M3 = E4M3_, TPA = D1 == 1;
    static constexpr bool PAIRED = E4M3 && R <= 2;             // the fp16 rebuild of two slots a lane
    static constexpr uint32_t Q_HALF = HQ * DH * 2, KV_TILE = TK * DH * 2;
    // A unit is what a factor stage holds: US slots in NG layout groups (8 slots, or 16 when e4m3).
    static constexpr int US = TPA ? 4096 / DH : TK, NU = TK / US, NG = US / (E4M3 ? 16 : 8);
    // d1 = 8: blocks of 8 elements x the unit's slots (A_r, then (r, hb) of B), then 32 scale bytes a
    // group.  d1 = 1: per group the B rows of every rank and the scale rows (contiguous in the pool as
    // h2 = 1: one copy), then (group, r) rows of A.
    static constexpr int BOX = NG * 128, NBLK = R * (1 + HB), FACT = NBLK * BOX;
    static constexpr int GROUP = R * D2 * 16 + (E4M3 ? 32 : 0), OFF_A = NG * GROUP;
    static constexpr int ST = TPA ? (OFF_A + NG * R * 16 + 127) / 128 * 128 : FACT + (E4M3 ? NG * 32 : 0);
    // factor stages of a plane: as many as fit beside the Q, K and V tiles (four at most)
    static constexpr size_t OFF_Q = 0;                         // two halves
    static constexpr size_t OFF_K = OFF_Q + 2 * Q_HALF;        // a buffer of K, and the third one
    static constexpr size_t OFF_V = OFF_K + 2 * KV_TILE;       // one buffer
    static constexpr size_t OFF_KST = OFF_V + KV_TILE;
    static constexpr size_t ROOM = 227 * 1024 - 256 - 1024 - 512 - OFF_KST;    // (static memory, alignment, barriers)
    static constexpr int FST = ROOM >= 8 * (size_t)ST && TPA ? 4 : ROOM >= 4 * (size_t)ST ? 2 : 1;
    static constexpr size_t OFF_VST = OFF_KST + (size_t)FST * ST;
    static constexpr size_t OFF_BAR = OFF_VST + (size_t)FST * ST;
    static constexpr int NBAR = 36;
    static constexpr size_t SMEM = 1024 + OFF_BAR + NBAR * 8 + 16;
    static_assert(TPA || D2 == 16 || (D2 == 8 && R == 2), "the fragment mapping covers d2 = 16, and 8 at R = 2");
    static_assert(!TPA || ((DH == 64 || DH == 128) && NG * R <= 32), "a unit's copies, one per lane");
    static_assert(ST % 16 == 0 && (TPA || ST % 128 == 0) && OFF_BAR % 8 == 0 && SMEM <= 227 * 1024 - 256, "shared memory");
};

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// Low word of a shared-memory descriptor (umma_desc_k_sw128's address and leading offset); the
// high word is the same for every tile.
__device__ __forceinline__ uint32_t umma_lo(uint32_t smem_addr) { return ((smem_addr >> 4) & 0x3FFFu) | (1u << 16); }
constexpr uint32_t kUmmaHi = (1024u >> 4) | (1u << 14) | (2u << 29);

// D[tmem] (+)= A B^T with A in shared memory, or in tensor memory; issued by one thread.
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "r"(kUmmaHi)
        : "memory");
}
__device__ __forceinline__ void umma_ts_lo(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "r"(kUmmaHi)
        : "memory");
}

// The eight softmax warps wait for one another.
__device__ __forceinline__ void softmax_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxWarps * 32) : "memory");
}

// mbarrier slots
enum : int {
    B_Q = 0,
    B_QREADY = 1,      // +h
    B_K_FULL = 3,      // +buffer
    B_K_EMPTY = 5,
    B_V_FULL = 7,      // +buffer
    B_V_EMPTY = 9,
    B_S_FULL = 11,     // +h
    B_P_HALF = 13,     // +h: the first half of P's columns
    B_P_FULL = 15,     // +h
    B_O_FINAL = 17,    // +h
    B_DRAIN = 19,
    B_KST_FULL = 20,   // +stage
    B_VST_FULL = 24,
    B_KST_EMPTY = 28,
    B_VST_EMPTY = 32,
};

// What the two halves work on.  With more than 128 rows each half has its own rows and takes
// every local tile from 0 to its last.  With fewer both have the same rows and take turns on the
// tiles (alt): step i of half h is tile 2 i + h.
struct TilePlan {
    bool alt;
    int steps0, steps1;                           // of each half
    int n_kt;                                     // tiles of the CTA
    __device__ int steps(int h) const { return h ? steps1 : steps0; }
    __device__ bool active(int h, int i) const { return i < steps(h); }
    __device__ int tile(int h, int i) const { return alt ? 2 * i + h : i; }
    __device__ bool first_half(int h, int i) const { return alt || h == (active(0, i) ? 0 : 1); }    // on its tile
    __device__ bool last_half(int h, int i) const { return alt || h == (active(1, i) ? 1 : 0); }
    // The K and V buffers of a tile and how often each was used before.  There are three, and with alt a
    // fourth in the place of the query rows 128 .. 255 that there are not.
    bool k_two, v_two;
    __device__ int k_buf(int t) const { return k_two ? t & 1 : 0; }
    __device__ int k_use(int t) const { return k_two ? t >> 1 : t; }
    __device__ int v_buf(int t) const { return v_two ? t & 1 : 0; }
    __device__ int v_use(int t) const { return v_two ? t >> 1 : t; }
};

template <class C>
__global__ void __launch_bounds__(kThreads, 1)
paged_prefill_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ PrefillArgsP a) {
    constexpr int D1 = C::D1, R = C::R, DH = C::DH;
    [[maybe_unused]] constexpr int HB = C::HB;
    constexpr bool E4M3 = C::E4M3;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t bar0 = smem_u32(smem + C::OFF_BAR);
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_BAR + C::NBAR * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) tma_prefetch_desc(&tmq);
    const int head = blockIdx.x, split = blockIdx.y;                // (the parts of the longest tiles start first)
    const int h = a.h1 * a.h2, i1 = head / a.h2, i2 = head % a.h2;
    const uint64_t limit = a.wait_limit_ns;

    // ---- this CTA's rows: rows row0 .. row0 + n - 1 at positions pos0 + r
    const Found f = find_tile<2 * HQ, true>(blockIdx.z, a.p.cu, a.p.start, a.p.batch, a.p.n_rows, a.p.err);
    if (f.b < 0) return;
    const int b = f.b, q0 = f.i * 2 * HQ;
    const int row0 = f.r0 + q0, n = min(2 * HQ, f.n - q0);
    const long long pos0 = (long long)f.pos + q0;
    if (tid == 0 && (pos0 < 0 || pos0 + n > a.p.max_len)) raise_error(a.p.err, kErrDeviceCheck);

    // ---- tiles: what the rows with a position in [0, max_len) see
    const int lo = (int)max(pos0, 0ll), hi = (int)min(pos0 + n - 1, (long long)a.p.max_len - 1);
    Tiles tl = {0, 0, 0};
    if (lo <= hi) tl = visible_tiles(a.p.mask, lo, hi, TK);
    const int wstart = lo <= hi ? window_start(a.p.mask, lo) : 0;
    int v0, v1;
    split_run(tl.n, split, a.p.n_split, v0, v1);
    TilePlan tp;
    tp.alt = n <= HQ;
    // The third buffer is K's second at d1 = 8, where the same warps rebuild K ahead of V.  At d1 = 1, where
    // V has its own warps and takes them longest, it is V's (d_h = 128, 9 x 256 rows over 4096 slots: 144 us
    // against 149).
    tp.k_two = !C::TPA || tp.alt;
    tp.v_two = C::TPA || tp.alt;
    auto own_steps = [&](int hh) {                 // tiles that the rows of a half see
        const long long plo = max(pos0 + hh * HQ, 0ll);
        const long long phi = min(pos0 + min(n, (hh + 1) * HQ) - 1, (long long)a.p.max_len - 1);
        return hh * HQ < n && plo <= phi ? max(min((int)(phi / TK) - tl.gap, v1 - 1) - v0 + 1, 0) : 0;
    };
    tp.steps0 = own_steps(0);
    tp.steps1 = own_steps(1);
    tp.n_kt = max(tp.steps0, tp.steps1);
    const bool q0_read = tp.steps0 > 0, q1_read = tp.steps1 > 0;          // which query rows are
    auto q_read = [&](int hh) { return hh ? q1_read : q0_read; };
    if (tp.alt) {
        tp.steps0 = (tp.n_kt + 1) / 2;
        tp.steps1 = tp.n_kt / 2;
    }
    constexpr uint32_t kThird = (uint32_t)(C::OFF_K + C::KV_TILE), kFourth = (uint32_t)(C::OFF_Q + C::Q_HALF);
    auto k_off = [&](int t) { return tp.k_buf(t) ? (C::TPA ? kFourth : kThird) : (uint32_t)C::OFF_K; };
    auto v_off = [&](int t) { return tp.v_buf(t) ? (C::TPA ? kThird : kFourth) : (uint32_t)C::OFF_V; };
    auto seen = [&](int s) { return s <= hi && (s >= wstart || s < a.p.mask.sinks); };

    // ---- producers' side (one warp per plane): page lookups and copies
    const bool is_producer = warp >= kProducerWarp, prod_v = warp == kProducerWarp + 1;
    // Pages are looked up for several units at a time (a load waited for at every unit would cost the warp
    // more than its copies): lane l holds run l % RUNS of unit u + l / RUNS.  A run is 16 slots at d1 = 8, a
    // group of the unit at d1 = 1.  in_page: its 16-slot group inside its page (-1: nothing, or seen by no
    // row).
    constexpr int RUNS = C::TPA ? C::NG : TK / 16, UNITS = 32 / RUNS;
    int page = 0, in_page = -1;
    auto fetch = [&](int u0) {
        in_page = -1;
        const int u = u0 + lane / RUNS, t = u / C::NU;
        if (t >= tp.n_kt) return;
        constexpr int span = C::TPA && !E4M3 ? 8 : 16;
        const int s0 = tl.slot_tile(v0 + t) * TK + (u % C::NU) * C::US + lane % RUNS * span;
        if (s0 > hi || (s0 + span <= wstart && s0 >= a.p.mask.sinks)) return;
        int entry;
        split_group(a.pool, s0 >> 4, entry, in_page);
        page = __ldg(a.pool.table + (size_t)b * a.pool.table_stride + entry);
    };
    // the head's factor slices of unit u (its pages looked up) into its stage, which is free
    auto copy_factors = [&](int u) {
        const int from = u % UNITS * RUNS + lane % RUNS;
        const int pu = __shfl_sync(0xffffffffu, page, from), iu = __shfl_sync(0xffffffffu, in_page, from);
        long long grp = -1;                                       // (lane < RUNS) the group of this lane's run
        if (lane < RUNS && iu >= 0) {
            const bool bad = pu < 0 || pu >= a.pool.n_pages;
            if (bad) raise_error(a.p.err, kErrDeviceCheck);
            grp = (long long)(bad ? 0 : pu) * a.pool.pg + iu;
        }
        const int s = u % C::FST;
        const uint32_t full = bar((prod_v ? B_VST_FULL : B_KST_FULL) + s);
        const uint32_t st = smem_u32(smem + (prod_v ? C::OFF_VST : C::OFF_KST) + (size_t)s * C::ST);
        const unsigned char *plane = prod_v ? a.pool.v : a.pool.k;
        const int gb = prod_v ? a.pool.vg : a.pool.kg;
        const int ab = R * a.h1 * D1;                             // first B element of a record
        if constexpr (C::TPA) {
            // The B rows as one bulk copy per group (each costs its warp about 100 clocks, one lane after the
            // other), the 16-byte A rows as plain asynchronous copies.
            const int loaded = __popc(__ballot_sync(0xffffffffu, grp >= 0));
            if (lane == 0) mbar_expect_tx(full, (uint32_t)loaded * C::GROUP);
            __syncwarp();
            auto half = [&](int g) { return !E4M3 && (g & 1) ? gb / 2 : 0; };      // of the two 8-slot groups of 16 slots
            if (grp >= 0) sm100::bulk_g2s(st + lane * C::GROUP, plane + grp * gb + half(lane) + ab * 16, C::GROUP, full);
            const long long ga = __shfl_sync(0xffffffffu, grp, lane / R % C::NG);
            if (lane < C::NG * R && ga >= 0)
                sm100::cp_async16(st + C::OFF_A + lane * 16,
                                  plane + ga * gb + half(lane / R) + ((lane % R) * a.h1 + i1) * 16);
        } else {
            // Runs of 8 rows of 16 bytes, four groups at a time: plain asynchronous copies, 24 instructions a
            // plane and tile at R = 2 in bf16 whatever the page size (a tensor copy per page and run costs the
            // warp about 130 clocks each: 96 of them at R = 4 and 16-slot pages).
            const int row = lane & 7;
#pragma unroll 1
            for (int g0 = 0; g0 < C::NG; g0 += 4) {
                const int g = g0 + (lane >> 3);
                const long long gg = __shfl_sync(0xffffffffu, grp, E4M3 ? g : g >> 1);
                const unsigned char *src = plane + gg * gb + (!E4M3 && (g & 1) ? gb / 2 : 0) + row * 16;
                const uint32_t dst = st + g * 128 + row * 16;
                if (gg >= 0) {
#pragma unroll
                    for (int k = 0; k < C::NBLK; ++k) {
                        const int e = k < R ? (k * a.h1 + i1) * D1
                                            : ab + (((k - R) / HB) * a.h2 + i2) * C::D2 + ((k - R) % HB) * 8;
                        sm100::cp_async16(dst + k * C::BOX, src + e * 16);
                    }
                }
            }
            if constexpr (E4M3) {                                 // the two scale rows of each group
                const long long gg = __shfl_sync(0xffffffffu, grp, lane >> 1 & 7);
                if (lane < 16 && gg >= 0) sm100::cp_async16(st + C::FACT + lane * 16, plane + gg * gb + gb - 32 + (lane & 1) * 16);
            }
        }
        sm100::cp_async_arrive(full);                             // every lane, for its own copies
    };
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    if (is_producer) fetch(0);
    if (warp == kProducerWarp) {
        // the first copies need none of the other warps: the query, then the first key factors
        if (lane == 0) {
            for (int i = 0; i < C::NBAR; ++i) {
                uint32_t count = 1;
                if ((i >= B_QREADY && i < B_QREADY + 2) || (i >= B_P_HALF && i < B_P_FULL + 2)) count = 4;
                if (i >= B_KST_FULL && i < B_KST_EMPTY) count = C::TPA ? 1 + 32 : 32;
                if (i >= B_KST_EMPTY || (i >= B_K_FULL && i < B_K_FULL + 2) || (i >= B_V_FULL && i < B_V_FULL + 2)) count = C::TPA ? kRebuildWarps / 2 : kRebuildWarps;
                mbar_init(bar(i), count);
            }
            *abort_flag = 0;
            mbar_fence_init();
            if (tp.n_kt > 0) {
                mbar_expect_tx(bar(B_Q), (uint32_t)((q0_read ? 1 : 0) + (q1_read ? 1 : 0)) * C::Q_HALF);
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
                    if (q_read(hh))
#pragma unroll
                        for (int cb = 0; cb < DH / 64; ++cb)
                            tma_load_2d(smem_u32(smem + C::OFF_Q + hh * C::Q_HALF + cb * HQ * 128), &tmq,
                                        head * DH + cb * 64, row0 + hh * HQ, bar(B_Q));
            }
        }
        __syncwarp();
    }
    if (warp == kProducerWarp && tp.n_kt > 0) copy_factors(0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // Bounded wait shared by every role: gives up when the time runs out or another thread has
    // already given up, and records the timeout once.
    auto wait = [&](int i, uint32_t parity) -> bool {
        if (mbar_try_wait(bar(i), parity)) return true;
        const uint64_t t0 = globaltimer();
        for (uint32_t it = 1;; ++it) {
            if (mbar_try_wait(bar(i), parity)) return true;
            if ((it & 15) == 0) {
                if (*abort_flag) return false;
                if (globaltimer() - t0 > limit) {
                    *abort_flag = 1;
                    raise_error(a.p.err, kErrTimeout);
                    return false;
                }
            }
        }
    };

    // The same by a whole warp: its lanes stay together, and the first polls do without the timer.
    auto wait_warp = [&](int i, uint32_t parity) -> bool {
        uint64_t t0 = 0;
        for (uint32_t it = 1;; ++it) {
            if (__all_sync(0xffffffffu, mbar_try_wait(bar(i), parity))) return true;
            if ((it & 15) == 0) {
                const uint64_t now = globaltimer();
                if (it == 16) t0 = now;
                const bool late = now - t0 > limit;
                if (late && lane == 0 && !*abort_flag) {
                    *abort_flag = 1;
                    raise_error(a.p.err, kErrTimeout);
                }
                if (__any_sync(0xffffffffu, late || *abort_flag)) return false;
            }
        }
    };

    if (is_producer) {
        // ---------------------------------------------------------------- producers
        if (tp.n_kt > 0) {
            const int b_empty = prod_v ? B_VST_EMPTY : B_KST_EMPTY, b_full = prod_v ? B_VST_FULL : B_KST_FULL;
            if (prod_v) copy_factors(0);
            int issued = 0;
            for (int u = 1; u < tp.n_kt * C::NU; ++u) {
                if (u % UNITS == 0) fetch(u);
                if (u >= C::FST && !wait_warp(b_empty + u % C::FST, ((u / C::FST) - 1) & 1)) break;
                copy_factors(u);
                issued = u;
            }
            // every copy this warp started lands before the CTA can exit
            if (!prod_v) (void)mbar_wait(bar(B_Q), 0, limit);
            for (int u = max(0, issued - C::FST + 1); u <= issued; ++u)
                (void)mbar_wait(bar(b_full + u % C::FST), (u / C::FST) & 1, limit);
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------- MMA issue
        if (lane == 0 && tp.n_kt > 0) {
            const uint32_t idesc_s = umma_idesc_f16_f32(HQ, TK), idesc_o = umma_idesc_f16_f32(HQ, DH);
            bool ok = true;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
                if (ok && q_read(hh) && !wait(B_QREADY + hh, 0)) ok = false;
            const uint32_t d_q = umma_lo(smem_u32(smem + C::OFF_Q)), d_0 = umma_lo(smem_u32(smem));
            // step i of half hh
            auto issue_s = [&](int hh, int i) -> bool {
                const int t = tp.tile(hh, i), kb = tp.k_buf(t);
                const uint32_t q_lo = tp.alt ? d_q : d_q + hh * (C::Q_HALF >> 4), k_lo = d_0 + (k_off(t) >> 4);
                const uint32_t s_addr = tmem + hh * 128;
                const bool last = tp.last_half(hh, i);
                if (!wait(B_K_FULL + kb, tp.k_use(t) & 1)) return false;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < DH / 16; ++k)
                    umma_ss(s_addr, q_lo + (k / 4) * (HQ * 128 >> 4) + 2 * (k % 4), k_lo + (k / 4) * (TK * 128 >> 4) + 2 * (k % 4),
                            idesc_s, k > 0);
                umma_commit(bar(B_S_FULL + hh));
                if (last) umma_commit(bar(B_K_EMPTY + kb));
                return true;
            };
            auto issue_pv = [&](int hh, int i) -> bool {
                const int t = tp.tile(hh, i), vb = tp.v_buf(t);
                const uint32_t v_lo = d_0 + (v_off(t) >> 4);
                const bool first = tp.first_half(hh, i), last = tp.last_half(hh, i), final = i == tp.steps(hh) - 1;
                if (!wait(B_P_HALF + hh, i & 1)) return false;
                if (first && !wait(B_V_FULL + vb, tp.v_use(t) & 1)) return false;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < TK / 16; ++k) {
                    if (k == TK / 32) {                               // the rest of P
                        if (!wait(B_P_FULL + hh, i & 1)) return false;
                        tc_fence_after();
                    }
                    umma_ts_lo(tmem + 256 + hh * 128, tmem + hh * 128 + 8 * k, v_lo + (k / 4) * (DH * 128 >> 4) + 2 * (k % 4), idesc_o,
                               i > 0 || k > 0);
                }
                if (last) umma_commit(bar(B_V_EMPTY + vb));
                if (final) umma_commit(bar(B_O_FINAL + hh));
                return true;
            };
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
                if (ok && tp.active(hh, 0)) ok = issue_s(hh, 0);
            for (int i = 0; i < max(tp.steps0, tp.steps1) && ok; ++i) {
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    if (ok && tp.active(hh, i)) ok = issue_pv(hh, i);
                    if (ok && tp.active(hh, i + 1)) ok = issue_s(hh, i + 1);
                }
            }
            // nothing issued here may still run when tensor memory is released
            umma_commit(bar(B_DRAIN));
            (void)mbar_wait(bar(B_DRAIN), 0, limit);
        }
    } else if (warp >= kRebuildWarp0) {
        // ---------------------------------------------------------------- K / V rebuild
        const int rw = warp - kRebuildWarp0;
        const int tok = lane >> 2;                 // slot of the 8-slot group this lane holds
        const int blk = lane >> 3, brow = lane & 7;   // ldmatrix / stmatrix row this lane addresses
        // Unit j of one plane of local tile t: K (slot rows, stmatrix) or V^T (feature rows, stmatrix.trans).
        auto rebuild = [&](int t, int j, auto v_c) {
            constexpr bool is_v = decltype(v_c)::value;
            const int fs = (t * C::NU + j) % C::FST;
            const unsigned char *st = smem + (is_v ? C::OFF_VST : C::OFF_KST) + (size_t)fs * C::ST;
            const uint32_t dst = smem_u32(smem) + (is_v ? v_off(t) : k_off(t));
            const int t0 = tl.slot_tile(v0 + t) * TK;
            const bool edge = !(t0 + TK - 1 <= hi && t0 >= wstart);
            // the exact fp16 scales of an e4m3 group's slots tok and tok + 8 (scale rows at e): half of each
            // token's exponent on A, half on B
            auto paired_scales = [&](const unsigned char *e, uint32_t &sa2, uint32_t &sb_lo, uint32_t &sb_hi) {
                const uint32_t ea = *reinterpret_cast<const uint16_t *>(e), eb = *reinterpret_cast<const uint16_t *>(e + 16);
                const int x0 = (int)(((ea & 255u) + (eb & 255u) + 130u) & 255u) - 128;
                const int x1 = (int)(((ea >> 8) + (eb >> 8) + 130u) & 255u) - 128;
                auto half_exp = [](int x) { return __uint_as_float((uint32_t)(127 + x) << 23); };
                sa2 = pack_half2(half_exp(x0 >> 1), half_exp(x1 >> 1));
                const float b0 = half_exp(x0 - (x0 >> 1)), b1 = half_exp(x1 - (x1 >> 1));
                sb_lo = pack_half2(b0, b0);
                sb_hi = pack_half2(b1, b1);
            };
            // four 8-feature blocks of 8-slot group g from feature f_first on: this lane's words w, its block's
            // first feature f0
            auto store_blocks = [&](int g, int f0, const uint32_t (&w)[4]) {
                if (!is_v)
                    stsm_x4(dst + (f0 >> 6) * (TK * 128) + sw128_chunk(g * kGroup + brow, (f0 & 63) >> 3), w[0], w[1], w[2], w[3]);
                else
                    stsm_x4_t(dst + (g >> 3) * (DH * 128) + sw128_chunk(f0 + brow, g & 7), w[0], w[1], w[2], w[3]);
            };
            if constexpr (C::TPA && !E4M3) {
                // two pieces of one 8-slot group and 64 features per warp
                constexpr int FP = 8 / C::NG;                      // pieces of a group
#pragma unroll
                for (int pc = 0; pc < 2; ++pc) {
                    const int at = 2 * (rw & 3) + pc, gu = at / FP, fp = at % FP, g = j * C::NG + gu;
                    const unsigned char *ga = st + C::OFF_A + gu * R * 16, *gb = st + gu * C::GROUP;
                    float av[R];
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        av[r] = __uint_as_float(
                            (uint32_t)(*reinterpret_cast<const uint16_t *>(ga + r * 16 + 2 * tok)) << 16);
                    const bool zero = edge && !seen(t0 + g * kGroup + tok);
#pragma unroll
                    for (int q4 = 0; q4 < 2; ++q4) {
                        const int f0 = fp * 64 + (q4 * 4 + blk) * 8;
                        float2 acc[4];
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            uint32_t bw[4];
                            ldsm_x4_t(smem_u32(gb + (r * C::D2 + f0 + brow) * 16), bw);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 a2 = make_float2(av[r], av[r]), x = unpack_bf16x2(bw[i]);
                                acc[i] = r == 0 ? fmul2(a2, x) : ffma2(a2, x, acc[i]);
                            }
                        }
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = zero ? 0u : pack_half2(acc[i].x, acc[i].y);
                        store_blocks(g, f0, w);
                    }
                }
                return;
            }
            if constexpr (C::TPA && E4M3) {
                // two pieces of one 16-slot group and 32 features per warp, slots tok and tok + 8 per lane (see below)
                constexpr int FP = 8 / C::NG;
#pragma unroll
                for (int pc = 0; pc < 2; ++pc) {
                    const int at = 2 * (rw & 3) + pc, gu = at / FP, fp = at % FP;
                    const int g = 2 * (j * C::NG + gu), f0 = fp * 32 + blk * 8;
                    const unsigned char *ga = st + C::OFF_A + gu * R * 16, *gb = st + gu * C::GROUP;
                    uint32_t sa2, sb_lo, sb_hi, w[2][4];
                    paired_scales(gb + C::GROUP - 32 + 2 * tok, sa2, sb_lo, sb_hi);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const uint32_t x =
                            hmul2(e4m3x2_to_h2(*reinterpret_cast<const uint16_t *>(ga + r * 16 + 2 * tok)), sa2);
                        const uint32_t a_lo = __byte_perm(x, 0, 0x1010), a_hi = __byte_perm(x, 0, 0x3232);
                        uint32_t bw[4];
                        ldsm_x4_t(smem_u32(gb + (r * C::D2 + f0 + brow) * 16), bw);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t lo2, hi2;
                            e4m3_split(bw[i], lo2, hi2);
                            lo2 = hmul2(lo2, sb_lo);
                            hi2 = hmul2(hi2, sb_hi);
                            w[0][i] = r == 0 ? hmul2(a_lo, lo2) : hfma2(a_lo, lo2, w[0][i]);
                            w[1][i] = r == 0 ? hmul2(a_hi, hi2) : hfma2(a_hi, hi2, w[1][i]);
                        }
                    }
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        if (edge && !seen(t0 + (g + hf) * kGroup + tok)) w[hf][0] = w[hf][1] = w[hf][2] = w[hf][3] = 0u;
                        store_blocks(g + hf, f0, w[hf]);
                    }
                }
                return;
            }
            if constexpr (C::PAIRED && !C::TPA) {
                // One 16-slot group per warp, slots tok and tok + 8 (neighbouring bytes) per lane, in
                // fp16: a code times half of its token's exponent is exact, so is the product of two
                // (2^-25 where it leaves fp16's normal range), and the sum over the two ranks is
                // rounded once.
                const int lg = rw;
                const unsigned char *grp = st + lg * 128, *e = st + C::FACT + lg * 32 + 2 * tok;
                uint32_t sa2, sb_lo, sb_hi;
                paired_scales(e, sa2, sb_lo, sb_hi);
                uint32_t bw[4], blo[4], bhi[4];                    // block r * HB + hb: features of tok, of tok + 8
                if constexpr (HB == 2) {
                    ldsm_x4_t(smem_u32(grp + (R + blk) * C::BOX + brow * 16), bw);
                } else {
                    uint32_t b2[2];
                    ldsm_x2_t(smem_u32(grp + (R + (blk & 1)) * C::BOX + brow * 16), b2);
                    bw[0] = b2[0], bw[1] = b2[1], bw[2] = bw[3] = 0u;
                }
#pragma unroll
                for (int i = 0; i < R * HB; ++i) {
                    e4m3_split(bw[i], blo[i], bhi[i]);
                    blo[i] = hmul2(blo[i], sb_lo);
                    bhi[i] = hmul2(bhi[i], sb_hi);
                }
                const bool zero_lo = edge && !seen(t0 + lg * 16 + tok), zero_hi = edge && !seen(t0 + lg * 16 + 8 + tok);
                constexpr int JN = 4 / HB;
#pragma unroll
                for (int i = 0; i < 8 / JN; ++i) {
                    uint32_t w[2][4];
#pragma unroll
                    for (int u = 0; u < JN; ++u) {
                        uint32_t a_lo[R], a_hi[R];
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const uint32_t x = hmul2(
                                e4m3x2_to_h2(*reinterpret_cast<const uint16_t *>(grp + r * C::BOX + (i * JN + u) * 16 + 2 * tok)), sa2);
                            a_lo[r] = __byte_perm(x, 0, 0x1010);
                            a_hi[r] = __byte_perm(x, 0, 0x3232);
                        }
#pragma unroll
                        for (int hb = 0; hb < HB; ++hb) {
                            const uint32_t lo2 = hfma2(a_lo[1], blo[HB + hb], hmul2(a_lo[0], blo[hb]));
                            const uint32_t hi2 = hfma2(a_hi[1], bhi[HB + hb], hmul2(a_hi[0], bhi[hb]));
                            w[0][u * HB + hb] = zero_lo ? 0u : lo2;
                            w[1][u * HB + hb] = zero_hi ? 0u : hi2;
                        }
                    }
                    const int f0 = HB == 2 ? (2 * i + (blk >> 1)) * 16 + (blk & 1) * 8 : (4 * i + blk) * 8;
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) store_blocks(2 * lg + hf, f0, w[hf]);
                }
                return;
            }
            if constexpr (C::TPA || C::PAIRED) return;
#pragma unroll 1
            for (int gi = 0; gi < TK / kGroup / kRebuildWarps; ++gi) {
                const int g = rw * (TK / kGroup / kRebuildWarps) + gi;        // 8-slot group of the tile
                const int lg = E4M3 ? g >> 1 : g, hf = g & 1;                 // its layout group, and half of it
                // A_r[tok][j1]: one 16-byte row per j1 holds the group's slots
                float av[R][8];
                if constexpr (E4M3) {
                    const unsigned char *e = st + C::FACT + lg * 32 + 2 * tok + hf;
                    const float sc = exp_sum(((uint32_t)e[0] + e[16] + 130u) & 255u);
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int j1 = 0; j1 < 8; ++j1)
                            av[r][j1] = h2_to_f2(e4m3x2_to_h2(st[r * C::BOX + lg * 128 + j1 * 16 + 2 * tok + hf])).x * sc;
                } else {
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int j1 = 0; j1 < 8; ++j1)
                            av[r][j1] = __uint_as_float(
                                (uint32_t)(*reinterpret_cast<const uint16_t *>(st + r * C::BOX + lg * 128 + j1 * 16 + tok * 2))
                                << 16);
                }
                // B_r[tok][hb*8 + 2c .. +1] for (r, hb) = block r * HB + hb
                constexpr int NB = R * HB;
                float2 bf[NB];
                auto unpack = [&](uint32_t w) {
                    if constexpr (E4M3) return h2_to_f2(e4m3x2_to_h2(__byte_perm(w, 0, hf ? 0x4431 : 0x4420)));
                    return unpack_bf16x2(w);
                };
                if constexpr (HB == 2) {
#pragma unroll
                    for (int q4 = 0; q4 < NB / 4; ++q4) {          // four blocks (two ranks) per load
                        uint32_t bw[4];
                        ldsm_x4_t(smem_u32(st + (R + 4 * q4 + blk) * C::BOX + lg * 128 + brow * 16), bw);
#pragma unroll
                        for (int i = 0; i < 4; ++i) bf[4 * q4 + i] = unpack(bw[i]);
                    }
                } else {
                    uint32_t bw[2];                                // lanes 0..15 address the two blocks
                    ldsm_x2_t(smem_u32(st + (R + (blk & 1)) * C::BOX + lg * 128 + brow * 16), bw);
#pragma unroll
                    for (int i = 0; i < 2; ++i) bf[i] = unpack(bw[i]);
                }
                uint32_t w[8][HB];
#pragma unroll
                for (int j1 = 0; j1 < 8; ++j1)
#pragma unroll
                    for (int hb = 0; hb < HB; ++hb) {
                        float2 acc = fmul2(make_float2(av[0][j1], av[0][j1]), bf[hb]);
#pragma unroll
                        for (int r = 1; r < R; ++r)
                            acc = ffma2(make_float2(av[r][j1], av[r][j1]), bf[r * HB + hb], acc);
                        w[j1][hb] = pack_half2(acc.x, acc.y);
                    }
                if (edge && !seen(t0 + g * kGroup + tok)) {
#pragma unroll
                    for (int j1 = 0; j1 < 8; ++j1)
#pragma unroll
                        for (int hb = 0; hb < HB; ++hb) w[j1][hb] = 0u;
                }
                // this lane addresses row brow of block blk of each x4 store: d2 = 16, (j1 = 2i +
                // blk/2, hb = blk%2); d2 = 8, j1 = 4i + blk
#pragma unroll
                for (int i = 0; i < 8 / (4 / HB); ++i) {
                    const int f0 = HB == 2 ? (2 * i + (blk >> 1)) * 16 + (blk & 1) * 8 : (4 * i + blk) * 8;
                    uint32_t w4[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) w4[k] = HB == 2 ? w[2 * i + (k >> 1)][(k & 1) * (HB - 1)] : w[(4 * i + k) & 7][0];
                    store_blocks(g, f0, w4);
                }
            }
        };
        // unit j of a plane of tile t: its factors landed, and (first unit) the products over the tile it
        // replaces done
        auto unit = [&](int t, int j, auto v_c) -> bool {
            constexpr bool is_v = decltype(v_c)::value;
            const int u = t * C::NU + j, fs = u % C::FST;                 // factor stage
            bool ok = true;
            if (j == 0 && !is_v && tp.k_use(t) >= 1) ok = wait_warp(B_K_EMPTY + tp.k_buf(t), (tp.k_use(t) - 1) & 1);
            if (j == 0 && is_v && tp.v_use(t) >= 1) ok = wait_warp(B_V_EMPTY + tp.v_buf(t), (tp.v_use(t) - 1) & 1);
            if (!ok || !wait_warp((is_v ? B_VST_FULL : B_KST_FULL) + fs, (u / C::FST) & 1)) return false;
            rebuild(t, j, v_c);
            if (j == C::NU - 1) fence_async_smem();         // visible to the tensor cores
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar((is_v ? B_VST_EMPTY : B_KST_EMPTY) + fs));
                if (j == C::NU - 1) mbar_arrive(bar(is_v ? B_V_FULL + tp.v_buf(t) : B_K_FULL + tp.k_buf(t)));
            }
            return true;
        };
        // the units of K of tile tk and of V of tile tv in turn (a plane's next copy lands while the
        // other plane's unit is rebuilt); a tile past the last, or below 0, is skipped
        auto both = [&](int tk, int tv) -> bool {
            bool ok = true;
#pragma unroll 1
            for (int j = 0; j < C::NU && ok; ++j) {         // (not unrolled: the roles share the instruction cache)
                if (tk < tp.n_kt) ok = unit(tk, j, std::false_type{});
                if (ok && tv >= 0) ok = unit(tv, j, std::true_type{});
            }
            return ok;
        };
        if constexpr (C::TPA) {
            // d1 = 1: four warps per plane (a unit is little work for eight)
            auto plane = [&](auto v_c) {
                bool ok = true;
#pragma unroll 1
                for (int u = 0; u < tp.n_kt * C::NU && ok; ++u) ok = unit(u / C::NU, u % C::NU, v_c);
            };
            if (rw < kRebuildWarps / 2)
                plane(std::false_type{});
            else
                plane(std::true_type{});
        } else {
            bool ok = tp.n_kt > 0;
            for (int t = -1; t < tp.n_kt && ok; ++t) ok = both(t + 1, t);
        }
    } else {
        // ---------------------------------------------------------------- softmax rows
        const int hh = warp >> 2, quarter = warp & 3;
        const int hq = tp.alt ? 0 : hh * HQ;                             // the half's first row
        const int row = quarter * 32 + lane, r = hq + row;
        const bool exists = r < n;
        const long long at = pos0 + r;
        const bool live = exists && at >= 0 && at < a.p.max_len;
        const size_t rh = (size_t)(row0 + r) * h + head;
        if (tp.steps(hh) > 0) {
            // Q_h: bf16 -> fp16 x qscale in place, once its copy has landed
            bool ok = true;
            if (q_read(hh)) ok = wait_warp(B_Q, 0);
            if (ok && q_read(hh)) {
                uint4 *q4 = reinterpret_cast<uint4 *>(smem + C::OFF_Q + hh * C::Q_HALF);
#pragma unroll 4
                for (int i = row; i < (int)(C::Q_HALF / 16); i += HQ) {
                    uint4 u = q4[i];
                    uint32_t *wv = reinterpret_cast<uint32_t *>(&u);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 x = unpack_bf16x2(wv[k]);
                        wv[k] = pack_half2(x.x * a.p.qscale, x.y * a.p.qscale);
                    }
                    q4[i] = u;
                }
                fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_QREADY + hh));

            const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
            const uint32_t s_addr = tmem + lane_off + hh * 128;
            const uint32_t o_addr = tmem + lane_off + 256 + hh * 128;
            const int pos = live ? (int)at : -1;                         // (-1 sees nothing)
            const int wlow = window_start(a.p.mask, pos);
            const int half_lo = (int)max(pos0 + hq, 0ll);                // smallest position of the half
            const int half_w = window_start(a.p.mask, (int)min(pos0 + min(n, hq + HQ) - 1, (long long)hi));
            const bool all_live = pos0 + hq >= 0 && pos0 + min(n, hq + HQ) <= a.p.max_len;
            float m_used = -INFINITY, l_run = 0.f;
            for (int i = 0; i < tp.steps(hh) && ok; ++i) {
                ok = wait_warp(B_S_FULL + hh, i & 1);
                if (!ok) break;
                tc_fence_after();
                const int t0 = tl.slot_tile(v0 + tp.tile(hh, i)) * TK;
                const bool masked = t0 + TK - 1 > half_lo || t0 < half_w || !all_live;
                // slots j <= lim of the tile, from low on or below sink, are visible
                const int lim = pos - t0, low = wlow - t0, sink = a.p.mask.sinks - t0;
                // the visible ones of slots 32 c .. 32 c + 31 as bits
                auto upto = [](int j) { return j < 0 ? 0u : j >= 31 ? 0xffffffffu : (2u << j) - 1u; };   // bits 0 .. j
                auto visible = [&](int c) {
                    return upto(lim - c * 32) & (~upto(low - 1 - c * 32) | upto(sink - 1 - c * 32));
                };
                float mx = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < TK / 32; ++c) {
                    float v[32];
                    tmem_ld32(s_addr + c * 32, v);
                    if (masked) {
                        const uint32_t vis = visible(c);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(vis >> j & 1u)) v[j] = -INFINITY;
                    }
                    float ma = fmax3(mx, v[0], v[1]), mb = fmax3(v[2], v[3], v[4]);
#pragma unroll
                    for (int j = 5; j < 29; j += 4) {
                        ma = fmax3(ma, v[j], v[j + 1]);
                        mb = fmax3(mb, v[j + 2], v[j + 3]);
                    }
                    mx = fmax3(ma, mb, fmax3(v[29], v[30], v[31]));
                }
                const bool grow = mx > m_used + kRescaleLog2;
                float alpha = 1.f;
                if (grow) {
                    alpha = m_used == -INFINITY ? 0.f : ex2(m_used - mx);
                    m_used = mx;
                    l_run *= alpha;
                }
                if (i > 0 && __any_sync(0xffffffffu, grow)) {
#pragma unroll 1
                    for (int c = 0; c < DH / 32; ++c) {
                        float v[32];
                        tmem_ld32(o_addr + c * 32, v);
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] *= alpha;
                        tmem_st32(o_addr + c * 32, v);
                    }
                }
                const float mref = m_used == -INFINITY ? 0.f : m_used;
                const float2 mref2 = make_float2(mref, mref);
                float2 suma = make_float2(0.f, 0.f), sumb = make_float2(0.f, 0.f);
#pragma unroll 1
                for (int c = 0; c < TK / 32; ++c) {
                    float v[32];
                    tmem_ld32(s_addr + c * 32, v);
                    uint32_t pw[16];
                    const uint32_t vis = masked ? visible(c) : 0xffffffffu;
#pragma unroll
                    for (int jp = 0; jp < 16; ++jp) {
                        const float2 x = fsub2(make_float2(v[2 * jp], v[2 * jp + 1]), mref2);
                        // one pair in four on the FMA pipe, the rest on the transcendental unit
                        float2 p = (jp & 3) == 3 ? exp2_poly2(x) : make_float2(ex2(x.x), ex2(x.y));
                        if (masked) {
                            if (!(vis >> (2 * jp) & 1u)) p.x = 0.f;
                            if (!(vis >> (2 * jp + 1) & 1u)) p.y = 0.f;
                        }
                        if (jp & 1)
                            sumb = fadd2(sumb, p);
                        else
                            suma = fadd2(suma, p);
                        pw[jp] = pack_half2(p.x, p.y);
                    }
                    tmem_st16u(s_addr + c * 16, pw);                  // P over the S columns already read
                    if (c == TK / 64 - 1) {                           // its products can start
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(B_P_HALF + hh));
                    }
                }
                l_run += (suma.x + suma.y) + (sumb.x + sumb.y);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_P_FULL + hh));
            }
            // epilogue: one row per thread, normalised or as this split's partial.  Halves that took turns
            // first join their maxima and sums (in a factor stage, whose last unit is long rebuilt); then each
            // writes half of the columns of both.
            const bool join = tp.alt && tp.steps1 > 0;
            if (ok) ok = wait_warp(B_O_FINAL + hh, 0);
            float m_row = m_used, l_row = l_run, w_own = 1.f, w_other = 0.f;
            if (join) {
                float2 *ml = reinterpret_cast<float2 *>(smem + C::OFF_KST);
                if (ok) ok = wait_warp(B_O_FINAL + (hh ^ 1), 0);
                if (ok) ml[hh * HQ + row] = make_float2(m_used, l_run);
                softmax_sync();
                ok = __all_sync(0xffffffffu, ok && !*abort_flag);
                const float2 o = ml[(hh ^ 1) * HQ + row];
                m_row = fmaxf(m_used, o.x);
                w_own = m_used == -INFINITY ? 0.f : ex2(m_used - m_row);
                w_other = o.x == -INFINITY ? 0.f : ex2(o.x - m_row);
                l_row = l_run * w_own + o.y * w_other;
            }
            const bool whole = a.p.n_split == 1;
            // Rows go out through the query tile, which no product reads any more: a thread's row is
            // strided by h d_h in memory, a row's 16-byte pieces by lanes are whole lines.
            constexpr int kRow = DH * 2;                                 // bytes of a bf16 row
            unsigned char *stage = smem + C::OFF_Q + hq * kRow + quarter * 32 * kRow;
            if (ok) {
                tc_fence_after();
                bool finite = true;
                const float inv = !whole ? 1.f : (l_row == 0.f ? 0.f : a.p.out_scale / l_row);
                if (!whole && exists && !(join && hh)) {
                    *reinterpret_cast<float2 *>(a.p.part_ml + (rh * a.p.n_split + split) * 2) =
                        make_float2(live ? m_row : -INFINITY, live ? l_row : 0.f);
                    finite = !live || (l_row <= 3.4e38f && m_row <= 3.4e38f);
                }
                w_own *= inv, w_other *= inv;
                const int c0 = join ? hh * (DH / 64) : 0, c1 = join ? c0 + DH / 64 : DH / 32;
#pragma unroll 1
                for (int c = c0; c < c1; ++c) {
                    float v[32];
                    tmem_ld32(o_addr + c * 32, v);
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] *= w_own;
                    if (join) {
#pragma unroll
                        for (int j0 = 0; j0 < 32; j0 += 16) {
                            float o[16];
                            sm100::tmem_ld16(tmem + lane_off + 256 + (hh ^ 1) * 128 + c * 32 + j0, o);
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j0 + j] += o[j] * w_other;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = live ? v[j] : 0.f;
                    if (exists) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) finite &= fabsf(v[j]) <= 3.4e38f;
                    }
                    if (whole) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
                            __nv_bfloat162 o2[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) o2[k] = __floats2bfloat162_rn(v[j + 2 * k], v[j + 2 * k + 1]);
                            const int piece = (c * 32 + j) / 8;          // rotated by the lane: no bank conflicts
                            *reinterpret_cast<uint4 *>(stage + lane * kRow + ((piece ^ (lane & 7)) << 4)) =
                                *reinterpret_cast<const uint4 *>(o2);
                        }
                    } else if (exists) {
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            *reinterpret_cast<float4 *>(a.p.part_o + (rh * a.p.n_split + split) * DH + c * 32 + j) =
                                make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                    }
                }
                if (!finite) raise_error(a.p.err, kErrDeviceCheck);
            }
            if (whole) {
                if (join)
                    softmax_sync();                                      // the other half's columns
                else
                    __syncwarp();
                constexpr int LPR = kRow / 16;                           // lanes per row
                const int piece = lane % LPR, first = quarter * 32 + hq;
                const int i0 = join ? hh * 16 : 0, i1 = join ? i0 + 16 : 32;     // this warp's rows of the quarter
#pragma unroll 4
                for (int i = i0 + lane / LPR; i < i1; i += 32 / LPR)
                    if (ok && first + i < n)
                        *reinterpret_cast<uint4 *>(a.p.out + ((size_t)(row0 + first + i) * h + head) * DH + piece * 8) =
                            *reinterpret_cast<const uint4 *>(stage + i * kRow + ((piece ^ (i & 7)) << 4));
            }
        } else if (exists && !(tp.alt && hh)) {                       // no tile of this half's rows here
            if (a.p.n_split > 1) {
                *reinterpret_cast<float2 *>(a.p.part_ml + (rh * a.p.n_split + split) * 2) = make_float2(-INFINITY, 0.f);
            } else {
                for (int c = 0; c < DH; c += 8)
                    *reinterpret_cast<uint4 *>(a.p.out + rh * DH + c) = make_uint4(0, 0, 0, 0);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <class C>
cudaError_t launch_cfg(const PagedShape &s, const PagedAttnArgs &p, unsigned long long wait_limit_ns, cudaStream_t st) {
    PrefillArgsP a;
    a.p = p;
    a.pool = s.pool;
    a.h1 = s.d.h1;
    a.h2 = s.d.h2;
    a.wait_limit_ns = wait_limit_ns;
    CUtensorMap tmq;
    if (!make_q_map(&tmq, p.q, (uint64_t)p.n_rows, (uint64_t)s.d.h * s.d.dh, HQ)) return cudaErrorInvalidValue;
    cudaError_t e = ensure_dynamic_smem<paged_prefill_kernel<C>>(C::SMEM);
    if (e != cudaSuccess) return e;
    const unsigned tiles = (unsigned)(((long long)p.n_rows + (long long)p.batch * (2 * HQ - 1)) / (2 * HQ));
    paged_prefill_kernel<C><<<dim3((unsigned)s.d.h, (unsigned)p.n_split, tiles), kThreads, C::SMEM, st>>>(tmq, a);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.n_split == 1) return e;
    return launch_paged_combine(s, p, st);
}

}  // namespace

int paged_prefill_rows() { return 2 * HQ; }

// The (d1, d2, R) of this repository's workloads that have equal R_K and R_V and rebuild a slot in the
// fragments above (any h1, and any h2 at d1 = 8).  The rest runs on mma.sync (4 x 4 heads of 4 x 16,
// R = 2, 8 x 2048 causal tokens: 675 us, 102 TFLOP/s).
bool paged_prefill_supported(const PagedShape &s) {
    const Dims &d = s.d;
    if (d.rk != d.rv) return false;
    if (d.d1 == 1) return d.h2 == 1 && ((d.d2 == 64 && d.rk <= 2) || (d.d2 == 128 && d.rk == 2));
    return d.d1 == 8 && ((d.d2 == 16 && (d.rk == 2 || d.rk == 4)) || (d.d2 == 8 && d.rk == 2));
}

cudaError_t launch_paged_prefill(const PagedShape &s, const PagedAttnArgs &a, unsigned long long wait_limit_ns,
                                 cudaStream_t st) {
    if (!paged_prefill_supported(s)) return cudaErrorInvalidValue;
    const Dims &d = s.d;
#define KPA_PREFILL_CASE(D1, D2, R)                                                             \
    if (d.d1 == D1 && d.d2 == D2 && d.rk == R)                                                  \
        return s.pool.e4m3 ? launch_cfg<Cfg<D1, D2, R, true>>(s, a, wait_limit_ns, st)          \
                           : launch_cfg<Cfg<D1, D2, R, false>>(s, a, wait_limit_ns, st);
    KPA_PREFILL_CASE(8, 16, 2)
    KPA_PREFILL_CASE(8, 16, 4)
    KPA_PREFILL_CASE(8, 8, 2)
    KPA_PREFILL_CASE(1, 64, 1)
    KPA_PREFILL_CASE(1, 64, 2)
    KPA_PREFILL_CASE(1, 128, 2)
#undef KPA_PREFILL_CASE
    return cudaErrorInvalidValue;
}

}  // namespace kpa
