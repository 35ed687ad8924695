// kpa_paged_decode.cu -- single-token attention over a paged factor cache on the tensor
// cores, for the head splits of KPA_PAGED_DECODE_VARIANTS (every other one runs on the
// chunk kernel).
//
// Proposition 2.2 of "Kronecker Product Attention" with a dense query, per 16-slot group:
//   T_r[(i1,j1), s] = sum_j2 q[(i1,i2),(j1,j2)] B^K_r(s)[i2,j2]         (mma.sync m16n8k16)
//   score[(i1,i2), s] = sum_r sum_j1 A^K_r(s)[i1,j1] T_r[(i1,j1), s]
//   O_i2[(i1,j1), j2] += sum_{s,r} (p[(i1,i2), s] A^V_r(s)[i1,j1]) B^V_r(s)[i2,j2]
// One warp takes 16 slots of one i2.  The query is an operand as it is over a bf16 pool, and over
// an e4m3 one (whose codes are exact in fp16) fp16 times a power of two of the warp's own, so
// the score products run once.  p A^V is rounded once by 2^-11 relative: to tf32 over a bf16 pool, whose B^V goes
// into the product as it is (fp16 operands lose factors of ordinary products but unequal
// magnitudes; they took 1 to 6 % less time: 8 x 4096 tokens of 4 x 8 heads of 8 x 16, R = 2,
// 17.2 us against 18.2, 64 x 4096 102 against 107), to fp16 over an e4m3 one.  Sums, scores
// and the softmax are fp32.  With d1 = 8 the rows of an m-tile pair up two j1 of one head per lane, so the
// sum over j1 is one add and two shuffles; with d1 = 1 (TPA) rows are heads.
//
// An e4m3 token's two key scales multiply its score (one number per token: the scales of a
// Kronecker product's factors multiply), its two value scales its B^V in fp16, times 2^8 that
// the output takes back, as far as codes up to 448 and down to 2^-3 stay exact there, and its
// weight beyond that: all products up to 2^22, with their precision down to 2^-16 (of the
// token's largest |A| |B|).
//
// Data movement: 16-slot groups are contiguous in the pool, so a run of them that the page table
// leaves together is one cp.async.bulk per plane into a ring of STAGES tiles; the last warp to
// release a stage issues its next tile, all warps the first ring.  The table entries of that tile are fetched while the current one is
// computed.  Only groups with a visible slot are copied; the slots of such a group that the
// query does not see are masked in the scores and zeroed in the value operands, so their
// bytes may hold anything.  Waits are bounded.
//
// Bound by instructions: 2^19 tokens of 4 x 8 heads of 8 x 16, R = 2, in e4m3 in 155 us (2.2 TB/s,
// 67 % of the issue slots); 32 ragged sequences at R = 4 in bf16 in 87 us (3.6 TB/s; tensor pipe
// 32 %); by latency on short ones: 8 x 4096 tokens of 16 heads of 64 in 11.7 us.
#include "kpa_f32x2.cuh"
#include "kpa_paged.cuh"
#include "kpa_sm100.cuh"

#include <cooperative_groups.h>

#include <type_traits>

namespace cg = cooperative_groups;

namespace kpa {
namespace {

using namespace paged;
using f32x2::ffma2;
using f32x2::fmul2;
using f32x2::unpack_bf16x2;
using sm100::bulk_g2s;
using sm100::mbar_expect_tx;
using sm100::mbar_init;
using sm100::mbar_wait;
using sm100::smem_u32;

struct DecodeArgsP {
    PagedAttnArgs p;
    Pool pool;
    int gps;                      // 16-slot groups per split (the blocks find it, with p.slots)
    int n_slots;                  // blocks, with p.slots
    int cluster;                  // the splits of a sequence are one cluster and merge over shared memory
    unsigned long long limit_ns;
    int skip_tile, skip_split;    // (tests) a tile of a split of sequence 0 that is never copied, or -1
};

// MA = h1*d1 rows of the products of one i2, SLICES token slices per CTA, HS warps that share
// a slice's 16-row tiles, CHUNKS groups per warp and tile, STAGES tiles in the ring.
template <int MA_, int D1_, int D2_, int RK_, int RV_, int H2_, int SLICES_, int HS_, int CHUNKS_, int STAGES_, bool Q8_>
struct Cfg {
    static constexpr int MA = MA_, D1 = D1_, D2 = D2_, RK = RK_, RV = RV_, H2 = H2_;
    static constexpr int SLICES = SLICES_, HS = HS_, CHUNKS = CHUNKS_, STAGES = STAGES_;
    static constexpr bool Q8 = Q8_, KPA = D1 == 8;
    static constexpr int H1 = MA / D1, H = H1 * H2, DH = D1 * D2;
    static constexpr int EK = RK * (MA + H2 * D2), EV = RV * (MA + H2 * D2);
    static constexpr int KG = Q8 ? (EK + 2) * 16 : EK * 32, VG = Q8 ? (EV + 2) * 16 : EV * 32;
    static constexpr int WARPS = H2 * SLICES * HS, THREADS = WARPS * 32;
    static constexpr int TG = SLICES * CHUNKS;                     // groups per tile
    static constexpr int STAGE_BYTES = TG * (KG + VG);
    static constexpr int MT = MA / 16 / HS;                        // 16-row tiles of a warp
    static constexpr int HR = KPA ? 1 : 2;                         // heads of a lane per tile
    static constexpr int MO_LD = DH + 8;                           // padded rows of the slice merge
    static constexpr size_t OFF_BARS = (size_t)STAGES * STAGE_BYTES;
    static constexpr size_t OFF_TAB = OFF_BARS + 8 * STAGES;                         // group indices of the next tiles
    // [0] abort, [1 + s] releases of stage s, [1 + STAGES + s] the last tile issued into it
    static constexpr size_t OFF_FLAGS = OFF_TAB + 8 * STAGES * TG;
    static constexpr size_t SMEM = OFF_FLAGS + 4 * (1 + 2 * STAGES);
    static_assert(MA % (16 * HS) == 0 && (KPA || (D1 == 1 && H2 == 1)) && (!KPA || HS == 1), "shape");
    static_assert(D2 % 16 == 0 || (KPA && D2 == 8), "d2");
    static constexpr int OFF_V = TG * KG;                          // a stage: the tile's K groups, then its V groups
    static constexpr int FIRST = (STAGES * TG + WARPS - 1) / WARPS;           // groups of the first ring per warp
    static_assert(WARPS <= 16 && TG <= 32 && FIRST <= 32, "one warp issues a tile");
    static_assert((size_t)(SLICES * H * (MO_LD + 2) + H * (DH + 2)) * 4 <= (size_t)STAGES * STAGE_BYTES,
                  "slice merge and merged partial fit in the ring");
    static_assert(SMEM <= 226 * 1024, "shared memory (a little is static)");
};

__device__ __forceinline__ void ldsm(uint32_t addr, uint32_t *r, std::integral_constant<int, 4>, std::false_type) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm(uint32_t addr, uint32_t *r, std::integral_constant<int, 4>, std::true_type) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm(uint32_t addr, uint32_t *r, std::integral_constant<int, 2>, std::false_type) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
}
__device__ __forceinline__ void ldsm(uint32_t addr, uint32_t *r, std::integral_constant<int, 2>, std::true_type) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
}
// N 8 x 8 matrices, matrix j's row `lane & 7` at row_of(j) * 16 bytes behind base
template <int N, bool TRANS, class RowOf>
__device__ __forceinline__ void ldsm_list(uint32_t base, int lane, uint32_t (&w)[N], RowOf row_of) {
    static_assert(N % 4 == 0 || N == 2, "matrices in fours, or two");
    if constexpr (N == 2) {
        ldsm(base + row_of((lane >> 3) & 1) * 16, w, std::integral_constant<int, 2>{}, std::bool_constant<TRANS>{});
    } else {
#pragma unroll
        for (int j = 0; j < N; j += 4)
            ldsm(base + row_of(j + (lane >> 3)) * 16, w + j, std::integral_constant<int, 4>{}, std::bool_constant<TRANS>{});
    }
}

template <bool F16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool F16>
__device__ __forceinline__ void mma8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(b0));
    else
        asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(b0));
}

__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// a float whose upper 19 bits, which a tf32 operand is, are x rounded to nearest (2^-11 relative); a NaN
// does not stay one (conversions that keep it take 7 to 17 % of the kernel)
__device__ __forceinline__ uint32_t to_tf32(float x) { return __float_as_uint(x) + 0x1000u; }

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// max as two bf16s, NaN where either is
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm volatile("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t mask_pair(uint32_t v, bool k0, bool k1) {
    return (k0 ? (v & 0xffffu) : 0u) | (k1 ? (v & 0xffff0000u) : 0u);
}
// SLOTS: the blocks size the splits themselves (a.p.slots).
template <class C, bool SLOTS>
__global__ void __launch_bounds__(C::THREADS, 1) paged_decode_kernel(const DecodeArgsP a) {
    constexpr int MA = C::MA, D1 = C::D1, D2 = C::D2, RK = C::RK, RV = C::RV, H2 = C::H2, H = C::H, DH = C::DH;
    constexpr int MT = C::MT, HR = C::HR, NT = D2 / 8, KS = D2 == 8 ? 1 : D2 / 16;
    constexpr int TG = C::TG, STAGES = C::STAGES, WARPS = C::WARPS, CHUNKS = C::CHUNKS, SLICES = C::SLICES, HS = C::HS;
    constexpr int KG = C::KG, VG = C::VG, A_K = RK * MA, A_V = RV * MA;
    constexpr bool Q8 = C::Q8, KPA = C::KPA;
    [[maybe_unused]] constexpr bool TURNS = H2 >= 4;       // (bf16) the warps of a slice share the look for NaN
    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t full0 = smem_u32(smem + C::OFF_BARS);
    size_t *tab = reinterpret_cast<size_t *>(smem + C::OFF_TAB);
    volatile int *flags = reinterpret_cast<volatile int *>(smem + C::OFF_FLAGS);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    const int i2 = warp % H2, hs = (warp / H2) % HS, slice = warp / (H2 * HS);

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) mbar_init(full0 + 8 * s, 1);
        for (int i = 0; i < 1 + STAGES; ++i) flags[i] = 0;
        for (int s = 0; s < STAGES; ++s) flags[1 + STAGES + s] = s;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    // ---- splits sized here: the smallest number of tiles P per split with which all sequences' splits
    // fit the blocks, so that one long sequence among short ones still loads every SM alike
    __shared__ int place[3];                               // sequence, split, groups per split
    if constexpr (SLOTS) {
        if (warp == 0) {
            constexpr int K = kPagedMaxSlotSeqs / 32;
            int tiles[K], sum = 0, most = 1;               // of sequences lane + 32 k
#pragma unroll
            for (int k = 0; k < K; ++k) {
                tiles[k] = 0;
                if (32 * k >= a.p.batch) continue;
                const int s = lane + 32 * k;
                const int n = s < a.p.batch ? min(a.p.seq_len[s], a.p.max_len) : 0;
                tiles[k] = n > 0 ? (visible_tiles(a.p.mask, n - 1, n - 1, 16).n + TG - 1) / TG : 0;
                sum += tiles[k];
                most = max(most, tiles[k]);
            }
            sum = (int)__reduce_add_sync(0xffffffffu, (unsigned)sum);
            most = (int)__reduce_max_sync(0xffffffffu, (unsigned)most);
            const int blocks = (int)gridDim.x;             // (at least one per sequence)
            int lo = max(1, sum / blocks), hi = most;      // hi does: one split per sequence
            while (lo < hi) {
                const int mid = lo + (hi - lo) / 2;
                int n = 0;
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (32 * k < a.p.batch) n += (int)((unsigned)(tiles[k] + mid - 1) / (unsigned)mid);
                if ((int)__reduce_add_sync(0xffffffffu, (unsigned)n) <= blocks)
                    hi = mid;
                else
                    lo = mid + 1;
            }
            // this block's sequence and split, in sequence order
            int before = 0, mine = -1, first = 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (32 * k >= a.p.batch) break;
                const int n = (int)((unsigned)(tiles[k] + hi - 1) / (unsigned)hi);
                int inc = n;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, inc, off);
                    if (lane >= off) inc += v;
                }
                const int at = before + inc - n;
                if (blockIdx.x == 0 && lane + 32 * k < a.p.batch) a.p.slots[lane + 32 * k] = make_int2(at, n);
                if ((int)blockIdx.x >= at && (int)blockIdx.x < at + n) mine = lane + 32 * k, first = at;
                before += __shfl_sync(0xffffffffu, inc, 31);
            }
            if (lane == 0) place[0] = -1;
            __syncwarp();
            if (mine >= 0) place[0] = mine, place[1] = (int)blockIdx.x - first, place[2] = hi * TG;
            // (a bad length is reported by its first split's block; one without a split, here)
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (blockIdx.x == 0 && lane + 32 * k < a.p.batch && a.p.seq_len[lane + 32 * k] < 0)
                    raise_error(a.p.err, kErrDeviceCheck);
        }
        __syncthreads();
        if (place[0] < 0) return;
    }
    const int b = SLOTS ? place[0] : (int)blockIdx.y, split = SLOTS ? place[1] : (int)blockIdx.x;
    const int gps = SLOTS ? place[2] : a.gps;
    // ---- this CTA's groups: virtual groups v0 .. v1 - 1 of the sequence's visible ones
    const int32_t *trow = a.pool.table + (size_t)b * a.pool.table_stride;
    int len = a.p.seq_len[b];
    // without a window the first ring's table entries do not depend on the length: fetch them
    // beside it (inside the row for every slot below max_len)
    const int v0 = split * gps;
    int first_page = 0, first_in = 0;
    const bool early = a.p.mask.window == 0, first_ring = lane < C::FIRST && warp * C::FIRST + lane < STAGES * TG;
    const int first_group = v0 + warp * C::FIRST + lane;
    if (first_ring && early && (long long)first_group * 16 < a.p.max_len) {
        int entry;
        split_group(a.pool, first_group, entry, first_in);
        first_page = __ldg(trow + entry);
    }
    // query fragments (A operand): row g (g + 8) of tile mt is (i1, j1) = (2 mt + (g >> 2), 2 (g & 3)) and
    // (i1, j1 + 1) with d1 = 8, head 16 mt + g (+ 8) with d1 = 1
    uint32_t qa[MT][KS][4];
    {
        const uint32_t *qb = reinterpret_cast<const uint32_t *>(a.p.q + (size_t)b * H * DH);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int v = 0; v < (D2 == 8 ? 2 : 4); ++v) {
                    const int j2 = ks * 16 + 2 * c + ((v & 2) ? 8 : 0);
                    int f;
                    if constexpr (KPA)
                        f = ((2 * mt + (g >> 2)) * H2 + i2) * DH + (2 * (g & 3) + (v & 1)) * D2 + j2;
                    else
                        f = ((hs * MT + mt) * 16 + g + 8 * (v & 1)) * DH + j2;
                    qa[mt][ks][v] = __ldg(qb + f / 2);
                }
    }
    if (len < 0 || len > a.p.max_len) {
        if (split == 0 && tid == 0) raise_error(a.p.err, kErrDeviceCheck);
        len = len < 0 ? 0 : a.p.max_len;
    }
    const int pos = len - 1;
    Tiles tl = {0, 0, 0};
    if (len > 0) tl = visible_tiles(a.p.mask, pos, pos, 16);
    const int wstart = len > 0 ? window_start(a.p.mask, pos) : 0;
    const int v1 = min(tl.n, v0 + gps);
    float *mo = reinterpret_cast<float *>(smem), *mm = mo + SLICES * H * C::MO_LD;      // (after the loop)
    float *merged = mm + SLICES * H * 2;                   // [H][DH] o, [H] m, [H] l: this CTA's, for its cluster
    // the cluster's partials joined: each CTA a run of the outputs.  Every CTA of a cluster comes here.
    auto join_cluster = [&] {
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();
        const int n_cl = a.p.n_split, per = (H * DH / 4 + n_cl - 1) / n_cl;
        const int lo = split * per, hi = min(H * DH / 4, lo + per);
        for (int i4 = lo + tid; i4 < hi; i4 += C::THREADS) {
            const int head = i4 * 4 / DH;
            float M = -INFINITY;
            for (int r = 0; r < n_cl; ++r) M = fmaxf(M, cl.map_shared_rank(merged, r)[H * DH + head]);
            float l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int r = 0; r < n_cl; ++r) {
                const float *rp = cl.map_shared_rank(merged, r);
                const float m = rp[H * DH + head], rl = rp[H * DH + H + head];
                if (m == -INFINITY && rl == 0.f) continue;
                const float w = exp2f(m - M);
                const float4 v = reinterpret_cast<const float4 *>(rp)[i4];
                l += w * rl;
                acc.x += w * v.x;
                acc.y += w * v.y;
                acc.z += w * v.z;
                acc.w += w * v.w;
            }
            const float f = l == 0.f ? 0.f : a.p.out_scale / l;
            __nv_bfloat162 w2[2] = {__floats2bfloat162_rn(acc.x * f, acc.y * f), __floats2bfloat162_rn(acc.z * f, acc.w * f)};
            *reinterpret_cast<uint2 *>(a.p.out + (size_t)b * H * DH + i4 * 4) = *reinterpret_cast<const uint2 *>(w2);
        }
        cl.sync();                                         // peers read this CTA's shared memory
    };
    auto partial_at = [&](int head) -> size_t {
        return SLOTS ? (size_t)blockIdx.x * H + head : (size_t)(b * H + head) * a.p.n_split + split;
    };
    auto empty_partial = [&] {
        for (int i = tid; i < H; i += C::THREADS) {
            if (a.cluster) {
                merged[H * DH + i] = -INFINITY;
                merged[H * DH + H + i] = 0.f;
            } else {
                *reinterpret_cast<float2 *>(a.p.part_ml + partial_at(i) * 2) = make_float2(-INFINITY, 0.f);
            }
        }
        if (a.cluster) join_cluster();
    };
    if (v0 >= v1) {                                        // nothing here: zeros, or an empty partial
        if (a.p.n_split == 1) {
            for (int i = tid; i < H * DH; i += C::THREADS)
                a.p.out[(size_t)b * H * DH + i] = __float2bfloat16_rn(0.f);
        } else {
            empty_partial();
        }
        return;
    }
    const int n_tiles = (v1 - v0 + TG - 1) / TG;
    __syncthreads();                                       // barriers initialised

    auto group_index = [&](int page, int in) -> size_t {
        if (page < 0 || page >= a.pool.n_pages) {
            raise_error(a.p.err, kErrDeviceCheck);
            page = 0;
        }
        return (size_t)page * a.pool.pg + in;
    };
    // Each lane's group (has) into place `at` of a stage, by a whole warp whose lanes hold places in order.
    // Groups that follow one another in the pool go as one copy per plane: a warp issues its lanes' copies
    // one after the other, about 100 clocks each.
    auto copy_groups = [&](int stage, int at, bool has, size_t group) {
        const size_t before = __shfl_up_sync(0xffffffffu, (unsigned long long)group, 1);
        const uint32_t heads = __ballot_sync(0xffffffffu, !has || lane == 0 || at == 0 || group != before + 1);
        if (has && (heads >> lane & 1u)) {
            const uint32_t later = lane == 31 ? 0u : heads >> (lane + 1);
            const uint32_t len = later ? __ffs(later) : 32 - lane;
            const uint32_t dst = smem_u32(smem) + stage * C::STAGE_BYTES;
            bulk_g2s(dst + at * KG, a.pool.k + group * KG, len * KG, full0 + 8 * stage);
            bulk_g2s(dst + C::OFF_V + at * VG, a.pool.v + group * VG, len * VG, full0 + 8 * stage);
        }
        __syncwarp();
    };
    auto groups_in = [&](int t) { return min(TG, v1 - v0 - t * TG); };
    auto withheld = [&](int t) { return t == a.skip_tile && split == a.skip_split && b == 0; };
    if (warp == 0 && lane < STAGES && lane < n_tiles && !withheld(lane)) mbar_expect_tx(full0 + 8 * lane, groups_in(lane) * (KG + VG));
    {                                                      // the first ring, some groups per warp
        const bool has = first_ring && first_group < v1 && !withheld((warp * C::FIRST + lane) / TG);
        if (has && !early) {
            int entry;
            split_group(a.pool, tl.slot_tile(first_group), entry, first_in);
            first_page = __ldg(trow + entry);
        }
        const int i = warp * C::FIRST + lane;
        copy_groups(i / TG, i % TG, has, has ? group_index(first_page, first_in) : 0);
    }

    // Over an e4m3 pool the query goes to fp16 times the power of two that takes the warp's largest
    // finite element to [2^14, 2^15): exact to 2^-31 of that element, off by at most 2^-39 of it below.  (Here: the first copies are on their way.)
    float qscale = a.p.qscale;
    if constexpr (Q8) {
        auto largest = [&](uint32_t limit) {               // largest bits of a magnitude up to limit
            uint32_t top = 0;
            auto take = [&](uint32_t bits) { top = max(top, bits <= limit ? bits : 0u); };
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int v = 0; v < (D2 == 8 ? 2 : 4); ++v) {
                        take(qa[mt][ks][v] & 0x7fffu);
                        take((qa[mt][ks][v] >> 16) & 0x7fffu);
                    }
            return __reduce_max_sync(0xffffffffu, top);
        };
        uint32_t top = largest(0x7fffu);
        if (top >= 0x7f80u) top = largest(0x7f7fu);        // (an element is not finite)
        top >>= 7;                                         // its exponent, biased by 127
        const uint32_t up = min(268u - top, 253u);         // that of the power
        const float scale = exp_byte(up);
        qscale *= exp_byte(254u - up);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int v = 0; v < (D2 == 8 ? 2 : 4); ++v) {
                    const float2 x = fmul2(unpack_bf16x2(qa[mt][ks][v]), make_float2(scale, scale));
                    qa[mt][ks][v] = pack_h2(x.x, x.y);
                }
    }
    float o[MT][NT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
    float m_run[MT][HR], l_run[MT][HR];                    // running max and this lane's share of the sum
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hr = 0; hr < HR; ++hr) {
            m_run[mt][hr] = -INFINITY;
            l_run[mt][hr] = 0.f;
        }
    uint32_t top_av = 0;                                   // the largest bf16 A^V of this thread, or NaN (which products lose)
    bool aborted = false;

    // rows (16 bytes each) of matrix j's fragments inside a group
    const int mrow = lane & 7;
    auto a_row = [&](int j) {                              // j = (r, mt, half)
        const int r = j / (2 * MT), mt = (j / 2) % MT, hf = j & 1;
        if constexpr (KPA) return r * MA + (2 * mt + (mrow >> 2)) * D1 + 2 * (mrow & 3) + hf;
        return r * MA + (hs * MT + mt) * 16 + hf * 8 + mrow;
    };
    auto b_row = [&](int j) {                              // j = (r, 8 features)
        return (j / NT) * H2 * D2 + i2 * D2 + (j % NT) * 8 + mrow;
    };

    for (int t = 0; t < n_tiles; ++t) {
        const int s = t % STAGES;
        // the table entries of the tile that follows in this stage, by one warp per tile
        const bool fetch = warp == t % WARPS && lane < TG && v0 + (t + STAGES) * TG + lane < v1;
        int next_page = 0, next_in = 0;
        if (fetch) {
            int entry;
            split_group(a.pool, tl.slot_tile(v0 + (t + STAGES) * TG + lane), entry, next_in);
            next_page = __ldg(trow + entry);
        }
        // (a vote: a warp whose lanes differ, as the time runs out, must not part)
        if (!__all_sync(0xffffffffu, mbar_wait(full0 + 8 * s, (t / STAGES) & 1, a.limit_ns))) {
            if (lane == 0) raise_error(a.p.err, kErrTimeout);
            flags[0] = 1;
            aborted = true;
            break;
        }
        const uint32_t stage = smem_u32(smem) + s * C::STAGE_BYTES;
        const int ng = groups_in(t), g0 = slice * CHUNKS;

        // NC groups from group gi0 of the tile on, with one softmax update.  MASKED: one group
        // with slots that the query does not see
        auto groups = [&](auto masked_c, auto nc_c, const int gi0) {
            constexpr bool MASKED = decltype(masked_c)::value;
            constexpr int NC = decltype(nc_c)::value;
            bool keep[2][2] = {{true, true}, {true, true}};        // slots 8 hf + 2c, + 1
            if constexpr (MASKED) {
                const int s0 = tl.slot_tile(v0 + t * TG + gi0) * 16 + 2 * c;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int sl = s0 + 8 * hf + u;
                        keep[hf][u] = sl <= pos && (sl >= wstart || sl < a.p.mask.sinks);
                    }
            }
            // ---- scores of this lane's heads, slots 2c, 2c + 1 of both halves
            float2 sc[NC][MT][HR][2];
#pragma unroll
            for (int cc = 0; cc < NC; ++cc) {
                const uint32_t kgrp = stage + (gi0 + cc) * KG;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int hr = 0; hr < HR; ++hr) sc[cc][mt][hr][0] = sc[cc][mt][hr][1] = make_float2(0.f, 0.f);
                uint32_t ew[2][RK * 2 * MT];                       // A^K words: [0] of both halves when e4m3
                if constexpr (Q8) {
                    ldsm_list<RK * 2 * MT, false>(kgrp, lane, ew[0], a_row);
                } else {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
                        ldsm_list<RK * 2 * MT, false>(kgrp + hf * (C::EK * 16), lane, ew[hf], a_row);
                }
#pragma unroll
                for (int r = 0; r < RK; ++r) {
                    float acc[MT][2][4];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
                            acc[mt][hf][0] = acc[mt][hf][1] = acc[mt][hf][2] = acc[mt][hf][3] = 0.f;
                    constexpr int STEP = NT >= 4 ? 4 : 2;          // matrices per load
                    if constexpr (D2 == 8) {
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            // one matrix a rank: lanes 0..7 address it (the pair load takes r and r again)
                            uint32_t bw[2];
                            if (Q8 && hf) break;
                            ldsm_list<2, true>(kgrp + A_K * 16 + (Q8 ? 0 : hf * (C::EK * 16)), lane, bw,
                                               [&](int) { return b_row(r); });
                            uint32_t b0 = bw[0], b1 = 0;
                            if constexpr (Q8) e4m3_split(bw[0], b0, b1);
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                mma8<Q8>(acc[mt][hf], qa[mt][0][0], qa[mt][0][1], b0);
                                if constexpr (Q8) mma8<Q8>(acc[mt][1], qa[mt][0][0], qa[mt][0][1], b1);
                            }
                        }
                    } else {
#pragma unroll
                        for (int n0 = 0; n0 < NT; n0 += STEP) {
#pragma unroll
                            for (int hf = 0; hf < (Q8 ? 1 : 2); ++hf) {
                                uint32_t bw[STEP];
                                ldsm_list<STEP, true>(kgrp + A_K * 16 + hf * (C::EK * 16), lane, bw,
                                                      [&](int j) { return b_row(r * NT + n0 + j); });
#pragma unroll
                                for (int k = 0; k < STEP / 2; ++k) {
                                    if constexpr (Q8) {
                                        uint32_t lo0, hi0, lo1, hi1;
                                        e4m3_split(bw[2 * k], lo0, hi0);
                                        e4m3_split(bw[2 * k + 1], lo1, hi1);
#pragma unroll
                                        for (int mt = 0; mt < MT; ++mt) {
                                            mma16<true>(acc[mt][0], qa[mt][n0 / 2 + k], lo0, lo1);
                                            mma16<true>(acc[mt][1], qa[mt][n0 / 2 + k], hi0, hi1);
                                        }
                                    } else {
#pragma unroll
                                        for (int mt = 0; mt < MT; ++mt)
                                            mma16<false>(acc[mt][hf], qa[mt][n0 / 2 + k], bw[2 * k], bw[2 * k + 1]);
                                    }
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int rh = 0; rh < 2; ++rh) {
                            float2 av[2];
                            const int j = (r * MT + mt) * 2 + rh;
                            if constexpr (Q8) {
                                uint32_t lo, hi;
                                e4m3_split(ew[0][j], lo, hi);
                                av[0] = h2_to_f2(lo);
                                av[1] = h2_to_f2(hi);
                            } else {
                                av[0] = unpack_bf16x2(ew[0][j]);
                                av[1] = unpack_bf16x2(ew[1][j]);
                            }
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                float2 &x = sc[cc][mt][KPA ? 0 : rh][hf];
                                x = ffma2(make_float2(acc[mt][hf][2 * rh], acc[mt][hf][2 * rh + 1]), av[hf], x);
                            }
                        }
                }
            }
            if constexpr (KPA) {                                   // the rest of the sum over j1: lanes that differ in g & 3
#pragma unroll
                for (int off = 4; off <= 8; off <<= 1)
#pragma unroll
                    for (int cc = 0; cc < NC; ++cc)
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                sc[cc][mt][0][hf].x += __shfl_xor_sync(0xffffffffu, sc[cc][mt][0][hf].x, off);
                                sc[cc][mt][0][hf].y += __shfl_xor_sync(0xffffffffu, sc[cc][mt][0][hf].y, off);
                            }
            }
            // ---- scale and mask
#pragma unroll
            for (int cc = 0; cc < NC; ++cc) {
                float2 ts[2] = {make_float2(qscale, qscale), make_float2(qscale, qscale)};
                if constexpr (Q8) {
                    const unsigned char *e = smem + s * C::STAGE_BYTES + (gi0 + cc) * KG + C::EK * 16 + 4 * c;
                    const uint32_t s4 = exp_sum4(*reinterpret_cast<const uint32_t *>(e), *reinterpret_cast<const uint32_t *>(e + 16));
                    // bytes: slots 2c, 2c + 8, 2c + 1, 2c + 9
                    ts[0] = make_float2(exp_sum(s4 & 255u) * qscale, exp_sum((s4 >> 16) & 255u) * qscale);
                    ts[1] = make_float2(exp_sum((s4 >> 8) & 255u) * qscale, exp_sum(s4 >> 24) * qscale);
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int hr = 0; hr < HR; ++hr)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            float2 &x = sc[cc][mt][hr][hf];
                            x = fmul2(x, ts[hf]);
                            if constexpr (MASKED) {
                                if (!keep[hf][0]) x.x = -INFINITY;
                                if (!keep[hf][1]) x.y = -INFINITY;
                            }
                        }
            }
            // ---- online softmax over the NC groups
            bool grow = false;
            float alpha[MT][HR];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int hr = 0; hr < HR; ++hr) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int cc = 0; cc < NC; ++cc)
                        mx = fmaxf(mx, fmaxf(fmaxf(sc[cc][mt][hr][0].x, sc[cc][mt][hr][0].y),
                                             fmaxf(sc[cc][mt][hr][1].x, sc[cc][mt][hr][1].y)));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    alpha[mt][hr] = 1.f;
                    if (mx > m_run[mt][hr]) {
                        alpha[mt][hr] = ex2(m_run[mt][hr] - mx);
                        m_run[mt][hr] = mx;
                        grow = true;
                    }
                    const float m = m_run[mt][hr];
                    float sum = 0.f;
#pragma unroll
                    for (int cc = 0; cc < NC; ++cc) {
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            sc[cc][mt][hr][hf].x = ex2(sc[cc][mt][hr][hf].x - m);
                            sc[cc][mt][hr][hf].y = ex2(sc[cc][mt][hr][hf].y - m);
                        }
                        sum += (sc[cc][mt][hr][0].x + sc[cc][mt][hr][0].y) + (sc[cc][mt][hr][1].x + sc[cc][mt][hr][1].y);
                    }
                    l_run[mt][hr] = l_run[mt][hr] * alpha[mt][hr] + sum;
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int v = 0; v < 4; ++v) o[mt][nt][v] *= alpha[mt][KPA ? 0 : v >> 1];
            }
            // ---- values
#pragma unroll
            for (int cc = 0; cc < NC; ++cc) {
                const uint32_t vgrp = stage + C::OFF_V + (gi0 + cc) * VG;
                uint32_t vs[2] = {0, 0}, p2[MT][HR][2];
                if constexpr (Q8) {
                    const unsigned char *e = smem + s * C::STAGE_BYTES + C::OFF_V + (gi0 + cc) * VG + C::EV * 16 + 4 * c;
                    const uint32_t s4 = exp_sum4(*reinterpret_cast<const uint32_t *>(e), *reinterpret_cast<const uint32_t *>(e + 16));
                    // 2^8 times the scales go to B while that is in [2^-18, 2^7] (bytes 102 .. 127): codes up to
                    // 448 then stay in fp16, and those down to 2^-3 stay exact.  What is beyond goes to the
                    // weights, for the whole warp at once (factors of standard deviation 2^-6 and less).
                    float2 f[2] = {make_float2(256.f * exp_sum(s4 & 255u), 256.f * exp_sum((s4 >> 16) & 255u)),
                                   make_float2(256.f * exp_sum((s4 >> 8) & 255u), 256.f * exp_sum(s4 >> 24))};
                    constexpr float kLow = 0x1p-18f, kHigh = 0x1p7f;
                    if (__any_sync(0xffffffffu, (((s4 & 0x7f7f7f7fu) + 0x1a1a1a1au) & ~s4 & 0x80808080u) != 0x80808080u)) {
                        auto within = [&](float x) { return fminf(fmaxf(x, kLow), kHigh); };
                        auto inverse = [](float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); };   // of a 2^k
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const float2 in = make_float2(within(f[hf].x), within(f[hf].y));
                            const float2 w = fmul2(f[hf], make_float2(inverse(in.x), inverse(in.y)));
                            f[hf] = in;
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                                for (int hr = 0; hr < HR; ++hr) sc[cc][mt][hr][hf] = fmul2(sc[cc][mt][hr][hf], w);
                        }
                    }
                    vs[0] = pack_h2(f[0].x, f[0].y);
                    vs[1] = pack_h2(f[1].x, f[1].y);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int hr = 0; hr < HR; ++hr)
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf)
                                p2[mt][hr][hf] = pack_h2(sc[cc][mt][hr][hf].x, sc[cc][mt][hr][hf].y);
                }
                uint32_t ew[2][RV * 2 * MT];
                if constexpr (Q8) {
                    ldsm_list<RV * 2 * MT, false>(vgrp, lane, ew[0], a_row);
                } else {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
                        ldsm_list<RV * 2 * MT, false>(vgrp + hf * (C::EV * 16), lane, ew[hf], a_row);
                    // Is an A^V a NaN?  The h2 warps of a slice hold the same ones: with four and more, each looks
                    // at its share (all of them by every warp: 4 % of the kernel at R = 4, the shares 1 %).
                    if constexpr (TURNS) {
                        constexpr int ALL = RV * 2 * MT, SHARE = 2 * ALL / H2, N = SHARE < 2 ? 2 : SHARE;
                        uint32_t w[N];
                        auto place = [&](int k) { return (i2 * SHARE + k) % (2 * ALL); };
                        ldsm_list<N, false>(vgrp, lane, w, [&](int k) { return a_row(place(k) % ALL) + place(k) / ALL * C::EV; });
#pragma unroll
                        for (int k = 0; k < N; ++k) {
                            const bool hf = place(k) >= ALL;
                            if constexpr (MASKED) w[k] = mask_pair(w[k], hf ? keep[1][0] : keep[0][0], hf ? keep[1][1] : keep[0][1]);
                            top_av = max_nan_bf16x2(top_av, w[k]);
                        }
                    } else if constexpr (MASKED) {
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                            for (int j = 0; j < RV * 2 * MT; ++j) {
                                ew[hf][j] = mask_pair(ew[hf][j], keep[hf][0], keep[hf][1]);
                                top_av = max_nan_bf16x2(top_av, ew[hf][j]);
                            }
                    }
                }
#pragma unroll
                for (int r = 0; r < RV; ++r) {
                    if constexpr (!Q8) {
                        // P' = p A^V_r as tf32, the bf16 B^V as it is: fp32's exponents, so that factors of any
                        // magnitudes keep P's 2^-11.  A half's eight slots are the k of one product: slot 2c at
                        // k = c and slot 2c + 1 at k = c + 4, in both operands.
                        uint32_t pt[2][MT][4];
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                                for (int rh = 0; rh < 2; ++rh) {
                                    const uint32_t w = ew[hf][(r * MT + mt) * 2 + rh];
                                    if constexpr (!MASKED && !TURNS) top_av = max_nan_bf16x2(top_av, w);
                                    const float2 x = fmul2(sc[cc][mt][KPA ? 0 : rh][hf], unpack_bf16x2(w));
                                    pt[hf][mt][rh] = !MASKED || !TURNS || keep[hf][0] ? to_tf32(x.x) : 0u;
                                    pt[hf][mt][2 + rh] = !MASKED || !TURNS || keep[hf][1] ? to_tf32(x.y) : 0u;
                                }
                        constexpr int STEP = NT >= 2 ? 2 : 1;          // 8-feature blocks per load
#pragma unroll
                        for (int n0 = 0; n0 < NT; n0 += STEP) {
                            // matrices (block, half): half 1 lies one 8-slot group further
                            uint32_t bw[2 * STEP];
                            ldsm_list<2 * STEP, false>(vgrp + A_V * 16, lane, bw, [&](int j) {
                                return b_row(r * NT + n0 + (j >> 1)) + (j & 1) * C::EV;
                            });
#pragma unroll
                            for (int k = 0; k < STEP; ++k)
#pragma unroll
                                for (int hf = 0; hf < 2; ++hf) {
                                    const uint32_t w = bw[2 * k + hf];
                                    const uint32_t b0 = !MASKED || keep[hf][0] ? w << 16 : 0u;
                                    const uint32_t b1 = !MASKED || keep[hf][1] ? w & 0xffff0000u : 0u;
#pragma unroll
                                    for (int mt = 0; mt < MT; ++mt) mma_tf32(o[mt][n0 + k], pt[hf][mt], b0, b1);
                                }
                        }
                    } else {
                        uint32_t pa[MT][4];                            // P' = p A^V_r: (half, rows g / g + 8)
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int rh = 0; rh < 2; ++rh) {
                                const int j = (r * MT + mt) * 2 + rh, hr = KPA ? 0 : rh;
                                uint32_t lo, hi;
                                e4m3_split(ew[0][j], lo, hi);
                                pa[mt][rh] = hmul2(p2[mt][hr][0], lo);
                                pa[mt][2 + rh] = hmul2(p2[mt][hr][1], hi);
                                if constexpr (MASKED) {
                                    pa[mt][rh] = mask_pair(pa[mt][rh], keep[0][0], keep[0][1]);
                                    pa[mt][2 + rh] = mask_pair(pa[mt][2 + rh], keep[1][0], keep[1][1]);
                                }
                            }
                        constexpr int STEP = NT >= 4 ? 4 : 2;          // 8-feature blocks per load
#pragma unroll
                        for (int n0 = 0; n0 < NT; n0 += STEP) {
                            uint32_t b0[STEP], b1[STEP];
                            uint32_t bw[STEP];
                            ldsm_list<STEP, false>(vgrp + A_V * 16, lane, bw, [&](int j) {
                                return b_row(r * NT + (NT == 1 ? 0 : n0 + j));
                            });
#pragma unroll
                            for (int k = 0; k < STEP; ++k) {
                                e4m3_split(bw[k], b0[k], b1[k]);
                                b0[k] = hmul2(b0[k], vs[0]);
                                b1[k] = hmul2(b1[k], vs[1]);
                            }
                            if constexpr (MASKED) {
#pragma unroll
                                for (int k = 0; k < STEP; ++k) {
                                    b0[k] = mask_pair(b0[k], keep[0][0], keep[0][1]);
                                    b1[k] = mask_pair(b1[k], keep[1][0], keep[1][1]);
                                }
                            }
#pragma unroll
                            for (int k = 0; k < STEP; ++k)
                                if (n0 + k < NT) {
#pragma unroll
                                    for (int mt = 0; mt < MT; ++mt) mma16<true>(o[mt][n0 + k < NT ? n0 + k : 0], pa[mt], b0[k], b1[k]);
                                }
                        }
                    }
                }
            }
        };
        // does group i of the tile hold slots that the query does not see?
        auto partial = [&](int i) {
            const int s0 = tl.slot_tile(v0 + t * TG + i) * 16;
            return s0 + 15 > pos || (s0 < wstart && s0 + 15 >= a.p.mask.sinks);
        };
        bool whole = g0 + CHUNKS <= ng;
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) whole = whole && !partial(g0 + i);
        if (whole) {
            groups(std::false_type{}, std::integral_constant<int, CHUNKS>{}, g0);
        } else {
#pragma unroll 1
            for (int i = 0; i < CHUNKS && g0 + i < ng; ++i) {
                if (CHUNKS == 1 || partial(g0 + i))
                    groups(std::true_type{}, std::integral_constant<int, 1>{}, g0 + i);
                else if constexpr (CHUNKS > 1)
                    groups(std::false_type{}, std::integral_constant<int, 1>{}, g0 + i);
            }
        }
        if (fetch) tab[s * TG + lane] = group_index(next_page, next_in);
        __syncwarp();
        // the last warp to release stage s issues tile t + STAGES into it (acq_rel: every
        // warp's reads of the stage, and the table entries, come first)
        uint32_t last = 0;
        if (lane == 0) {
            uint32_t old;
            asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;"
                         : "=r"(old)
                         : "r"(smem_u32((const void *)(flags + 1 + s)))
                         : "memory");
            last = (old + 1) % WARPS == 0 && t + STAGES < n_tiles && !flags[0] && !withheld(t + STAGES);
            if (last) {
                flags[1 + STAGES + s] = t + STAGES;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_expect_tx(full0 + 8 * s, groups_in(t + STAGES) * (KG + VG));
            }
        }
        last = __shfl_sync(0xffffffffu, last, 0);
        __syncwarp();                                       // lane 0's acquire covers the warp
        if (last) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            const int n = groups_in(t + STAGES);
            copy_groups(s, lane, lane < n, lane < n ? tab[s * TG + lane] : 0);
        }
        if (__any_sync(0xffffffffu, flags[0])) { aborted = true; break; }
    }
    __syncthreads();
    // Copies still in flight, of the last tile issued into each stage, land before the CTA ends or its
    // partial takes the ring's place.
    if (aborted || flags[0]) {
        if (tid < STAGES) {
            const int t = flags[1 + STAGES + tid];
            if (t < n_tiles && !withheld(t)) (void)mbar_wait(full0 + 8 * tid, (t / STAGES) & 1, a.limit_ns);
        }
        __syncthreads();
        if (a.p.n_split > 1) empty_partial();               // (the error is reported; peers must not wait)
        return;
    }

    // ---- the sum of each head over its lanes, then the merge of the token slices
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hr = 0; hr < HR; ++hr) {
            l_run[mt][hr] += __shfl_xor_sync(0xffffffffu, l_run[mt][hr], 1);
            l_run[mt][hr] += __shfl_xor_sync(0xffffffffu, l_run[mt][hr], 2);
        }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int rh = 0; rh < 2; ++rh) {
            const int head = KPA ? (2 * mt + (g >> 2)) * H2 + i2 : (hs * MT + mt) * 16 + g + 8 * rh;
            const int j1 = KPA ? 2 * (g & 3) + rh : 0, hr = KPA ? 0 : rh;
            float *dst = mo + (size_t)(slice * H + head) * C::MO_LD + j1 * D2;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                *reinterpret_cast<float2 *>(dst + nt * 8 + 2 * c) = make_float2(o[mt][nt][2 * rh], o[mt][nt][2 * rh + 1]);
            if (c == 0 && (!KPA || ((g & 3) == 0 && rh == 0)))
                *reinterpret_cast<float2 *>(mm + (slice * H + head) * 2) = make_float2(m_run[mt][hr], l_run[mt][hr]);
        }
    __syncthreads();
    constexpr float kBack = Q8 ? 1.f / 256.f : 1.f;
    bool finite = (top_av & 0x7fffu) <= 0x7f80u && (top_av >> 16 & 0x7fffu) <= 0x7f80u;
    for (int i4 = tid; i4 < H * DH / 4; i4 += C::THREADS) {
        const int head = i4 * 4 / DH, col = i4 * 4 % DH;
        float M = -INFINITY;
#pragma unroll
        for (int sl = 0; sl < SLICES; ++sl) M = fmaxf(M, mm[(sl * H + head) * 2]);
        float l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int sl = 0; sl < SLICES; ++sl) {
            const float2 ms = *reinterpret_cast<const float2 *>(mm + (sl * H + head) * 2);
            if (ms.x == -INFINITY && ms.y == 0.f) continue;         // a slice without a group
            const float w = exp2f(ms.x - M);
            const float4 v = *reinterpret_cast<const float4 *>(mo + (size_t)(sl * H + head) * C::MO_LD + col);
            l += w * ms.y;
            acc.x += w * v.x;
            acc.y += w * v.y;
            acc.z += w * v.z;
            acc.w += w * v.w;
        }
        const float f = a.p.n_split == 1 ? (l == 0.f ? 0.f : a.p.out_scale * kBack / l) : kBack;
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
        finite = finite && isfinite(acc.x) && isfinite(acc.y) && isfinite(acc.z) && isfinite(acc.w) && l <= 3.4e38f;
        if (a.p.n_split == 1) {
            __nv_bfloat162 w2[2] = {__floats2bfloat162_rn(acc.x, acc.y), __floats2bfloat162_rn(acc.z, acc.w)};
            *reinterpret_cast<uint2 *>(a.p.out + (size_t)b * H * DH + i4 * 4) = *reinterpret_cast<const uint2 *>(w2);
        } else if (a.cluster) {
            reinterpret_cast<float4 *>(merged)[i4] = acc;
            if (col == 0) {
                merged[H * DH + head] = M;
                merged[H * DH + H + head] = l;
            }
        } else {
            const size_t at = partial_at(head);
            *reinterpret_cast<float4 *>(a.p.part_o + at * DH + col) = acc;
            if (col == 0) *reinterpret_cast<float2 *>(a.p.part_ml + at * 2) = make_float2(M, l);
        }
    }
    // a cached value that is not finite, or an operand outside the fp16 range
    if (!finite) raise_error(a.p.err, kErrDeviceCheck);
    if (a.cluster) join_cluster();
}

// (variant, MA, D1, D2, RK, RV, H2, HS, then SLICES, CHUNKS, STAGES for bf16 and for e4m3 pools): the
// head splits of this repository's decode workloads whose i2 share the 16 warps of an SM evenly (h2
// a power of two) and whose h1 d1 is a multiple of 16.  h2 of 5 and 10 and h = 61 would need slices and padding of their own; they run on the chunk
// kernel, at its pace (4 x 5 heads of 8 x 8, R = 2, 8 x 4096 tokens: 275 us; 4 x 4 heads here: 16).
// Blocks are as large as an SM holds: smaller ones start sooner on short sequences and lose more on long
// ones (variant 0, bf16, 4 slices and 3 stages against 8 and 2: 8 x 4096 tokens 9.9 us against 10.7,
// 64 x 4096 53 against 45, 4 x 65536 57 against 35; variant 4, e4m3, 2 slices of 4 chunks against 8 of 2:
// 64 x 4096 25.8 against 25.1, 65536 37.3 against 16.7).
#define KPA_PAGED_DECODE_VARIANTS(X)            \
    X(0, 16, 1, 64, 2, 2, 1, 1, 8, 1, 2, 8, 2, 2)    \
    X(1, 32, 8, 16, 4, 4, 8, 1, 2, 1, 2, 2, 2, 2)    \
    X(2, 32, 8, 16, 2, 2, 8, 1, 2, 2, 2, 2, 2, 4)    \
    X(3, 32, 8, 16, 2, 2, 4, 1, 4, 1, 2, 4, 2, 2)    \
    X(4, 32, 1, 64, 1, 1, 1, 2, 4, 4, 2, 8, 2, 2)    \
    X(5, 32, 8, 8, 2, 2, 4, 1, 4, 2, 2, 4, 2, 2)     \
    X(6, 16, 8, 8, 2, 2, 8, 1, 2, 2, 2, 2, 2, 4)     \
    X(7, 64, 8, 8, 2, 2, 2, 1, 8, 1, 2, 8, 1, 2)     \
    X(8, 16, 1, 128, 2, 2, 1, 1, 4, 1, 2, 8, 1, 2)   \
    X(9, 32, 8, 16, 4, 4, 4, 1, 4, 1, 2, 4, 1, 4)

template <class C, bool SLOTS>
cudaError_t launch_cfg(const DecodeArgsP &a, cudaStream_t st) {
    cudaError_t e = ensure_dynamic_smem<paged_decode_kernel<C, SLOTS>>(C::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = SLOTS ? dim3((unsigned)a.n_slots) : dim3((unsigned)a.p.n_split, (unsigned)a.p.batch);
    lc.blockDim = dim3(C::THREADS);
    lc.dynamicSmemBytes = C::SMEM;
    lc.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster ? (unsigned)a.p.n_split : 1u;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 2;
    return cudaLaunchKernelEx(&lc, paged_decode_kernel<C, SLOTS>, a);
}

template <class C>
cudaError_t launch_split(const DecodeArgsP &a, cudaStream_t st) {
    return a.p.slots ? launch_cfg<C, true>(a, st) : launch_cfg<C, false>(a, st);
}

// Clusters of `size` CTAs that can be resident at once on the current device (0: none).
template <class C>
int max_clusters(int size) {
    if (ensure_dynamic_smem<paged_decode_kernel<C, false>>(C::SMEM) != cudaSuccess) return 0;
    if (size > 8 && cudaFuncSetAttribute(paged_decode_kernel<C, false>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
                        cudaSuccess)
        return 0;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)size);
    lc.blockDim = dim3(C::THREADS);
    lc.dynamicSmemBytes = C::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, paged_decode_kernel<C, false>, &lc) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

}  // namespace

int paged_decode_variant(const Dims &d) {
#define KPA_MATCH(IDX, MA, D1, D2, RK, RV, H2, HS, ...) \
    if (d.h1 * d.d1 == MA && d.d1 == D1 && d.d2 == D2 && d.rk == RK && d.rv == RV && d.h2 == H2) return IDX;
    KPA_PAGED_DECODE_VARIANTS(KPA_MATCH)
#undef KPA_MATCH
    return -1;
}

void paged_decode_shape(int variant, bool e4m3, int *tile_groups, int *ctas_per_sm) {
    size_t smem = 1;
    int threads = 1;
    switch (variant) {
#define KPA_SHAPE(IDX, MA, D1, D2, RK, RV, H2, HS, S0, C0, T0, S1, C1, T1)          \
    case IDX:                                                                        \
        if (e4m3) {                                                                  \
            using C = Cfg<MA, D1, D2, RK, RV, H2, S1, HS, C1, T1, true>;             \
            *tile_groups = C::TG, smem = C::SMEM, threads = C::THREADS;              \
        } else {                                                                     \
            using C = Cfg<MA, D1, D2, RK, RV, H2, S0, HS, C0, T0, false>;            \
            *tile_groups = C::TG, smem = C::SMEM, threads = C::THREADS;              \
        }                                                                            \
        break;
        KPA_PAGED_DECODE_VARIANTS(KPA_SHAPE)
#undef KPA_SHAPE
        default:
            *tile_groups = 1;
    }
    // 1 KB of shared memory a CTA is the system's; a warp holds up to 128 registers a thread
    const int by_smem = (int)(228 * 1024 / (smem + 1024)), by_warps = 512 / threads;
    *ctas_per_sm = by_smem < by_warps ? by_smem : by_warps;
    if (*ctas_per_sm < 1) *ctas_per_sm = 1;
}

int paged_decode_max_clusters(int variant, bool e4m3, int size) {
    // asked once per device, variant, format and size
    constexpr int kDevices = 64, kVariants = 10;
    static std::atomic<int> known[kDevices][kVariants][2][kPagedMaxCluster + 1];
    int dev = 0;
    if (size < 2 || size > kPagedMaxCluster || variant < 0 || variant >= kVariants || cudaGetDevice(&dev) != cudaSuccess ||
        dev < 0 || dev >= kDevices)
        return 0;
    std::atomic<int> &k = known[dev][variant][e4m3][size];
    if (k.load() == 0) {
        int n = 0;
        switch (variant) {
#define KPA_CLUSTERS(IDX, MA, D1, D2, RK, RV, H2, HS, S0, C0, T0, S1, C1, T1)                        \
    case IDX:                                                                                        \
        n = e4m3 ? max_clusters<Cfg<MA, D1, D2, RK, RV, H2, S1, HS, C1, T1, true>>(size)             \
                 : max_clusters<Cfg<MA, D1, D2, RK, RV, H2, S0, HS, C0, T0, false>>(size);           \
        break;
            KPA_PAGED_DECODE_VARIANTS(KPA_CLUSTERS)
#undef KPA_CLUSTERS
        }
        k.store(n > 0 ? n : -1);
    }
    return k.load() > 0 ? k.load() : 0;
}

cudaError_t launch_paged_decode(int variant, const PagedShape &s, const PagedAttnArgs &p, int groups_per_split,
                                int n_slots, bool cluster, unsigned long long wait_limit_ns, cudaStream_t st) {
    DecodeArgsP a;
    a.p = p;
    a.pool = s.pool;
    a.gps = groups_per_split;
    a.cluster = cluster;
    a.n_slots = n_slots;
    a.limit_ns = wait_limit_ns;
    device_skip_hook(&a.skip_tile, &a.skip_split);
    cudaError_t e = cudaErrorInvalidValue;
    switch (variant) {
#define KPA_CASE(IDX, MA, D1, D2, RK, RV, H2, HS, S0, C0, T0, S1, C1, T1)                              \
    case IDX:                                                                                           \
        e = s.pool.e4m3 ? launch_split<Cfg<MA, D1, D2, RK, RV, H2, S1, HS, C1, T1, true>>(a, st)        \
                        : launch_split<Cfg<MA, D1, D2, RK, RV, H2, S0, HS, C0, T0, false>>(a, st);      \
        break;
        KPA_PAGED_DECODE_VARIANTS(KPA_CASE)
#undef KPA_CASE
    }
    if (e != cudaSuccess || p.n_split == 1 || cluster) return e;
    return launch_paged_combine(s, p, st);
}

}  // namespace kpa
