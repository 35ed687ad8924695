// kpa_paged_mma.cu -- attention over a paged factor cache for any Kronecker split of order 2
// with d_h <= 128, on mma.sync: chunks of new tokens and single tokens.
//
// One CTA takes 128 query rows of one head of one sequence (8 warps x 16 rows) and walks the
// 64-slot tiles its rows see: those of the sinks and those of its windows, or, when few CTAs
// would run, one of n_split equal runs of them, whose partials a second kernel joins.
//   - all threads copy the head's slices of the next tile's factor records into a two-stage
//     ring (cp.async, 16-byte vectors of one element's slots), each 16-slot group through
//     the page table;
//   - the CTA rebuilds K_h and V_h = sum_r A_r (x) B_r of the tile in fp32, rounded once to
//     fp16, feature-major into shared memory ("Kronecker Product Attention", eq 4); an e4m3
//     token's two scales multiply into its A factors.  Slots that none of the CTA's rows
//     sees are written as zeros whatever the pool holds there;
//   - each warp forms S = Q K^T for its 16 rows on m16n8k16 (fp16 operands, fp32 sums),
//     masks it, runs the online softmax in registers and adds P V (P rounded to fp16, 2^-11
//     relative) into its fp32 output tile.
// Bound by the rebuild and its fragments' way through shared memory: 8 x 2048 causal tokens of
// 4 x 4 heads of 8 x 16, R = 2, in 1179 us (117 TFLOP/s), where the tcgen05 kernel takes 255.  A single
// token is one live row of the 128: 8 x 4096 tokens of 61 heads of 64, R = 1, in 804 us.
#include <cuda_fp16.h>

#include "kpa_f32x2.cuh"
#include "kpa_paged.cuh"
#include "kpa_sm100.cuh"

namespace kpa {
namespace {

using namespace paged;
using f32x2::ffma2;
using f32x2::fmul2;
using f32x2::unpack_bf16x2;
using sm100::cp_async16;
using sm100::smem_u32;

constexpr int kRows = 128;     // query rows per CTA
constexpr int kSlots = 64;     // key slots per tile
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

struct MmaArgs {
    PagedAttnArgs p;
    Pool pool;
    int h1, h2, d1, d2, dh, rk, rv;
    int ek, ev;                 // elements per key / value record
    int ekh, evh;               // one head's slice of a record, in elements (e4m3: and its two scale rows)
    int ekp, evp;               // stage stride of a group's slice, in 16-byte vectors (odd)
    int nch;                    // 4-column chunks of a B row: ceil(d2 / 4)
};

// Shared-memory layout (bytes): K tile, V tile (feature-major, 64 slots = 128 B per feature
// row), then a region that first holds Q and then the factor stages, and the table of a
// slice's rows inside a group.
struct Layout {
    int ks, vs, x, tab, total;
};

// groups of a tile: 8 slots each in bf16, 16 in e4m3
__host__ __device__ constexpr int tile_groups(bool e4m3) { return e4m3 ? kSlots / 16 : kSlots / 8; }

__host__ __device__ inline Layout layout_of(int DH, int ekh, int evh, int ekp, int evp, bool e4m3) {
    Layout L;
    L.ks = 0;
    L.vs = DH * 128;
    L.x = 2 * DH * 128;
    const int qb = kRows * DH * 2, sb = 2 * tile_groups(e4m3) * (ekp + evp) * 16;
    L.tab = L.x + (qb > sb ? qb : sb);
    L.total = L.tab + ((ekh + evh) * 4 + 15) / 16 * 16;
    return L;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// d += a b for one 16 x 8 x 16 tile: a row-major 16 x 16 fp16, b 16 x 8 fp16 (k pairs), d fp32
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8 slots of one element: bf16 pairs, or half hf of an e4m3 row (slot 8 hf + t at byte 2 t + hf)
template <bool E4M3>
__device__ __forceinline__ void unpack8(const uint4 v, int hf, float2 (&x)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
        x[k] = E4M3 ? h2_to_f2(e4m3x2_to_h2(__byte_perm(w[k], 0, hf ? 0x4431 : 0x4420))) : unpack_bf16x2(w[k]);
}

template <int DH, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1) paged_mma_kernel(const MmaArgs a) {
    static_assert(DH == 64 || DH == 128, "feature tile");
    constexpr int NC = DH / 8;        // 16-byte chunks of a Q row
    constexpr int KS = DH / 16;       // k-steps of Q K^T
    constexpr int G = tile_groups(E4M3), GS = kSlots / G;
    extern __shared__ __align__(128) unsigned char smem[];
    const Layout L = layout_of(DH, a.ekh, a.evh, a.ekp, a.evp, E4M3);
    unsigned char *Ks = smem + L.ks, *Vs = smem + L.vs, *X = smem + L.x;
    int *tab = reinterpret_cast<int *>(smem + L.tab);
    const int stage_bytes = G * (a.ekp + a.evp) * 16;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int head = blockIdx.x, split = blockIdx.z;
    const int h = a.h1 * a.h2, i1 = head / a.h2, i2 = head % a.h2;

    // ---- this CTA's rows: rows row0 .. row0 + n - 1, positions pos0 + r
    int b, row0, n;
    long long pos0;
    if (a.p.cu) {
        const Found f = find_tile<kRows>(blockIdx.y, a.p.cu, a.p.start, a.p.batch, a.p.n_rows, a.p.err);
        if (f.b < 0) return;
        b = f.b;
        row0 = f.r0 + f.i * kRows;
        n = min(kRows, f.n - f.i * kRows);
        pos0 = (long long)f.pos + f.i * kRows;
    } else {
        b = row0 = blockIdx.y;
        n = 1;
        int len = a.p.seq_len[b];
        if (len < 0 || len > a.p.max_len) {
            if (tid == 0) raise_error(a.p.err, kErrDeviceCheck);
            len = len < 0 ? 0 : a.p.max_len;
        }
        pos0 = len - 1;
    }
    // rows with a position in [0, max_len): lo .. hi; the others get zeros
    const int lo = (int)max(pos0, 0ll), hi = (int)min(pos0 + n - 1, (long long)a.p.max_len - 1);
    if (a.p.cu && tid == 0 && (pos0 < 0 || pos0 + n > a.p.max_len)) raise_error(a.p.err, kErrDeviceCheck);
    Tiles tl = {0, 0, 0};
    if (lo <= hi) tl = visible_tiles(a.p.mask, lo, hi, kSlots);
    int v0, v1;
    split_run(tl.n, split, a.p.n_split, v0, v1);
    const int wstart = lo <= hi ? window_start(a.p.mask, lo) : 0;
    // seen by some row of the CTA
    auto seen = [&](int s) { return s <= hi && (s >= wstart || s < a.p.mask.sinks); };

    // ---- prologue: slice table, zero feature rows d_h .. DH-1, Q tile
    for (int e = tid; e < a.ekh + a.evh; e += kThreads) {
        const bool v = e >= a.ekh;
        const int ee = v ? e - a.ekh : e, R = v ? a.rv : a.rk;
        int off;
        if (ee < R * a.d1)
            off = (ee / a.d1) * a.h1 * a.d1 + i1 * a.d1 + ee % a.d1;
        else if (ee < R * (a.d1 + a.d2)) {
            const int e2 = ee - R * a.d1;
            off = R * a.h1 * a.d1 + (e2 / a.d2) * a.h2 * a.d2 + i2 * a.d2 + e2 % a.d2;
        } else                                                   // e4m3: the two scale rows
            off = (v ? a.ev : a.ek) + ee - R * (a.d1 + a.d2);
        tab[e] = off;
    }
    for (int idx = tid; idx < (DH - a.dh) * 8 * 2; idx += kThreads) {
        const int row = a.dh + (idx >> 4), c = idx & 7;
        *reinterpret_cast<uint4 *>(((idx >> 3) & 1 ? Vs : Ks) + row * 128 + c * 16) = make_uint4(0, 0, 0, 0);
    }
    for (int idx = tid; idx < kRows * NC; idx += kThreads) {
        const int row = idx / NC, c = idx % NC, f0 = c * 8;
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (row < n && f0 < a.dh) {
            const uint32_t *src =
                reinterpret_cast<const uint32_t *>(a.p.q + ((size_t)(row0 + row) * h + head) * a.dh + f0);
#pragma unroll
            for (int p = 0; p < 4; ++p)
                if (f0 + 2 * p < a.dh) {
                    const float2 x = unpack_bf16x2(__ldg(src + p));
                    w[p] = pack_h2(x.x * a.p.qscale, x.y * a.p.qscale);
                }
        }
        *reinterpret_cast<uint4 *>(X + row * DH * 2 + ((c ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();
    // Q fragments of this warp's 16 rows, all k-steps, kept in registers
    uint32_t qa[KS][4];
    {
        const int row = warp * 16 + (lane & 15);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
            ldsm4(smem_u32(X + row * DH * 2 + (((2 * ks + (lane >> 4)) ^ (row & 7)) << 4)), qa[ks]);
    }
    __syncthreads();                                             // X becomes the factor stages

    // group g = tid % G of tile v, through the page table (null: seen by no row)
    const int my_g = tid % G;
    auto group_at = [&](int v, const unsigned char *&k, const unsigned char *&vv) {
        const int s0 = tl.slot_tile(v) * kSlots + my_g * GS;
        k = vv = nullptr;
        if (s0 > hi || (s0 + GS <= wstart && s0 >= a.p.mask.sinks)) return;
        int entry, in;
        split_group(a.pool, s0 >> 4, entry, in);
        int page = __ldg(a.pool.table + (size_t)b * a.pool.table_stride + entry);
        if (page < 0 || page >= a.pool.n_pages) {
            if (tid < G) raise_error(a.p.err, kErrDeviceCheck);
            page = 0;
        }
        const size_t g = (size_t)page * a.pool.pg + in;
        k = a.pool.k + g * a.pool.kg + (E4M3 ? 0 : (my_g & 1) * a.ek * 16);
        vv = a.pool.v + g * a.pool.vg + (E4M3 ? 0 : (my_g & 1) * a.ev * 16);
    };
    auto issue = [&](int stage, const unsigned char *k, const unsigned char *vv) {
        if (k) {
            unsigned char *st = X + stage * stage_bytes + my_g * a.ekp * 16;
            for (int e = tid / G; e < a.ekh; e += kThreads / G) cp_async16(smem_u32(st + e * 16), k + tab[e] * 16);
            unsigned char *sv = X + stage * stage_bytes + (G * a.ekp + my_g * a.evp) * 16;
            for (int e = tid / G; e < a.evh; e += kThreads / G)
                cp_async16(smem_u32(sv + e * 16), vv + tab[a.ekh + e] * 16);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    const int wrow0 = warp * 16;
    const bool warp_live = wrow0 < n;
    const long long pa_ = pos0 + wrow0 + (lane >> 2), pb_ = pa_ + 8;     // positions of this lane's two rows
    const bool ok0 = wrow0 + (lane >> 2) < n && pa_ >= 0 && pa_ < a.p.max_len;
    const bool ok1 = wrow0 + (lane >> 2) + 8 < n && pb_ >= 0 && pb_ < a.p.max_len;
    const int p0 = ok0 ? (int)pa_ : -1, p1 = ok1 ? (int)pb_ : -1;        // (-1 sees nothing)
    const int warp_hi = (int)min(pos0 + min(wrow0 + 15, n - 1), (long long)hi);
    const int warp_lo = (int)min(max(pos0 + wrow0, 0ll), (long long)INT32_MAX);
    const int warp_w = window_start(a.p.mask, warp_hi);
    float o[DH / 8][4];
#pragma unroll
    for (int nt = 0; nt < DH / 8; ++nt) o[nt][0] = o[nt][1] = o[nt][2] = o[nt][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    const int n_items = 8 * a.d1 * a.nch;                        // rebuild items per plane
    const unsigned char *nk = nullptr, *nv = nullptr;
    if (v0 < v1) {
        group_at(v0, nk, nv);
        issue(0, nk, nv);
        if (v0 + 1 < v1) group_at(v0 + 1, nk, nv);
    }
    for (int v = v0; v < v1; ++v) {
        const int cur = (v - v0) & 1;
        if (v + 1 < v1) {
            issue(cur ^ 1, nk, nv);
            if (v + 2 < v1) group_at(v + 2, nk, nv);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();                                         // stage landed; the tile before is fully used
        const int t0 = tl.slot_tile(v) * kSlots;

        // ---- rebuild K_h, V_h of the tile: item = (8-slot group g, row j1, 4 columns of B)
        {
            const uint4 *sk = reinterpret_cast<const uint4 *>(X + cur * stage_bytes);
            const uint4 *sv = sk + G * a.ekp;
            const bool edge = !(t0 + kSlots - 1 <= hi && t0 >= wstart);
            for (int it = tid; it < 2 * n_items; it += kThreads) {
                const bool isv = it >= n_items;
                const int i = isv ? it - n_items : it;
                const int g = i & 7, rest = i >> 3;
                const int j1 = rest / a.nch, c = rest - j1 * a.nch;
                const int R = isv ? a.rv : a.rk, gs = E4M3 ? g >> 1 : g, hf = g & 1;
                const uint4 *A = isv ? sv + gs * a.evp : sk + gs * a.ekp;
                const uint4 *B = A + R * a.d1;
                float2 acc[4][4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[u][k] = make_float2(0.f, 0.f);
                float2 sc[4];
                if constexpr (E4M3) {
                    const uint4 ea = A[R * (a.d1 + a.d2)], eb = A[R * (a.d1 + a.d2) + 1];
                    const uint32_t s4[4] = {exp_sum4(ea.x, eb.x), exp_sum4(ea.y, eb.y), exp_sum4(ea.z, eb.z),
                                            exp_sum4(ea.w, eb.w)};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        sc[k] = make_float2(exp_sum((s4[k] >> (8 * hf)) & 255u), exp_sum((s4[k] >> (16 + 8 * hf)) & 255u));
                }
                for (int r = 0; r < R; ++r) {
                    float2 av[4];
                    unpack8<E4M3>(A[r * a.d1 + j1], hf, av);
                    if constexpr (E4M3) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) av[k] = fmul2(av[k], sc[k]);
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int j2 = c * 4 + u;
                        if (j2 < a.d2) {
                            float2 x[4];
                            unpack8<E4M3>(B[r * a.d2 + j2], hf, x);
#pragma unroll
                            for (int k = 0; k < 4; ++k) acc[u][k] = ffma2(av[k], x[k], acc[u][k]);
                        }
                    }
                }
                unsigned char *dst = isv ? Vs : Ks;
                const int slot0 = t0 + g * 8;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int j2 = c * 4 + u;
                    if (j2 < a.d2) {
                        if (edge) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if (!seen(slot0 + 2 * k)) acc[u][k].x = 0.f;
                                if (!seen(slot0 + 2 * k + 1)) acc[u][k].y = 0.f;
                            }
                        }
                        const int f = j1 * a.d2 + j2;
                        *reinterpret_cast<uint4 *>(dst + f * 128 + ((g ^ (f & 7)) << 4)) =
                            make_uint4(pack_h2(acc[u][0].x, acc[u][0].y), pack_h2(acc[u][1].x, acc[u][1].y),
                                       pack_h2(acc[u][2].x, acc[u][2].y), pack_h2(acc[u][3].x, acc[u][3].y));
                    }
                }
            }
        }
        __syncthreads();                                         // K_h, V_h of the tile complete

        // no row of the warp sees the tile
        if (!warp_live || t0 > warp_hi ||
            (t0 + kSlots - 1 < window_start(a.p.mask, warp_lo) && t0 >= a.p.mask.sinks && a.p.mask.window > 0))
            continue;
        // ---- S = Q K^T (16 rows x 64 slots)
        float s[8][4];
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const int f = ks * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
            for (int np = 0; np < 4; ++np) {
                uint32_t kb[4];
                const int chunk = 2 * np + (lane >> 4);
                ldsm4_t(smem_u32(Ks + f * 128 + ((chunk ^ (f & 7)) << 4)), kb);
                mma_f16(s[2 * np], qa[ks], kb[0], kb[1]);
                mma_f16(s[2 * np + 1], qa[ks], kb[2], kb[3]);
            }
        }
        // ---- mask and online softmax (base 2: the scores carry log2 e)
        if (t0 + kSlots - 1 > warp_lo || t0 < warp_w || !ok0 || !ok1) {
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                const int j = t0 + nt * 8 + 2 * (lane & 3);
                if (!sees(a.p.mask, p0, j)) s[nt][0] = -INFINITY;
                if (!sees(a.p.mask, p0, j + 1)) s[nt][1] = -INFINITY;
                if (!sees(a.p.mask, p1, j)) s[nt][2] = -INFINITY;
                if (!sees(a.p.mask, p1, j + 1)) s[nt][3] = -INFINITY;
            }
        }
        float mx0 = m0, mx1 = m1;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            mx0 = fmaxf(mx0, fmaxf(s[nt][0], s[nt][1]));
            mx1 = fmaxf(mx1, fmaxf(s[nt][2], s[nt][3]));
        }
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
        const float ref0 = mx0 == -INFINITY ? 0.f : mx0, ref1 = mx1 == -INFINITY ? 0.f : mx1;
        const float al0 = m0 == -INFINITY ? 0.f : ex2f(m0 - ref0), al1 = m1 == -INFINITY ? 0.f : ex2f(m1 - ref1);
        m0 = mx0;
        m1 = mx1;
        float ps0 = 0.f, ps1 = 0.f;
        uint32_t pa[8][2];                                      // P as fp16 pairs, A-fragment order
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            const float e0 = ex2f(s[nt][0] - ref0), e1 = ex2f(s[nt][1] - ref0);
            const float e2 = ex2f(s[nt][2] - ref1), e3 = ex2f(s[nt][3] - ref1);
            ps0 += e0 + e1;
            ps1 += e2 + e3;
            pa[nt][0] = pack_h2(e0, e1);
            pa[nt][1] = pack_h2(e2, e3);
        }
        l0 = l0 * al0 + ps0;
        l1 = l1 * al1 + ps1;
#pragma unroll
        for (int nt = 0; nt < DH / 8; ++nt) {
            o[nt][0] *= al0;
            o[nt][1] *= al0;
            o[nt][2] *= al1;
            o[nt][3] *= al1;
        }
        // ---- O += P V
#pragma unroll
        for (int kk = 0; kk < kSlots / 16; ++kk) {
            const uint32_t pf[4] = {pa[2 * kk][0], pa[2 * kk][1], pa[2 * kk + 1][0], pa[2 * kk + 1][1]};
            const int chunk = 2 * kk + ((lane >> 3) & 1);
#pragma unroll
            for (int np = 0; np < DH / 16; ++np) {
                uint32_t vb[4];
                const int f = (2 * np + (lane >> 4)) * 8 + (lane & 7);
                ldsm4(smem_u32(Vs + f * 128 + ((chunk ^ (f & 7)) << 4)), vb);
                mma_f16(o[2 * np], pf, vb[0], vb[1]);
                mma_f16(o[2 * np + 1], pf, vb[2], vb[3]);
            }
        }
    }

    // ---- store the rows this warp owns: normalised, or this split's partial
    if (!warp_live) return;
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    bool finite = true;
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
        const int r = wrow0 + (lane >> 2) + 8 * hr;
        if (r >= n) continue;
        const bool ok = hr ? ok1 : ok0;
        const float l = hr ? l1 : l0, m = hr ? m1 : m0;
        const size_t rh = (size_t)(row0 + r) * h + head;
        if (a.p.n_split > 1) {
            const size_t at = rh * a.p.n_split + split;
            const bool any = ok && m > -INFINITY;                // (false for a NaN maximum: see below)
            const bool bad = ok && !(m <= 3.4e38f && l <= 3.4e38f);
            if ((lane & 3) == 0)
                *reinterpret_cast<float2 *>(a.p.part_ml + at * 2) = make_float2(ok ? m : -INFINITY, ok ? l : 0.f);
            finite = finite && !bad;
            if (!any && !bad) continue;
#pragma unroll
            for (int nt = 0; nt < DH / 8; ++nt) {
                const int f = nt * 8 + 2 * (lane & 3);
                if (f < a.dh) {
                    const float2 y = make_float2(o[nt][2 * hr], o[nt][2 * hr + 1]);
                    *reinterpret_cast<float2 *>(a.p.part_o + at * a.dh + f) = y;
                    finite = finite && isfinite(y.x) && isfinite(y.y);
                }
            }
        } else {
            const float inv = l == 0.f ? 0.f : a.p.out_scale / l;
#pragma unroll
            for (int nt = 0; nt < DH / 8; ++nt) {
                const int f = nt * 8 + 2 * (lane & 3);
                if (f < a.dh) {
                    const float2 y = ok ? make_float2(o[nt][2 * hr] * inv, o[nt][2 * hr + 1] * inv) : make_float2(0.f, 0.f);
                    *reinterpret_cast<__nv_bfloat162 *>(a.p.out + rh * a.dh + f) = __floats2bfloat162_rn(y.x, y.y);
                    finite = finite && isfinite(y.x) && isfinite(y.y);
                }
            }
        }
    }
    // a cached value that is not finite or outside the fp16 range makes rows non-finite
    if (!finite) raise_error(a.p.err, kErrDeviceCheck);
}

struct SliceDims {
    int DH, ekh, evh, ekp, evp;
};

SliceDims slice_dims(const Dims &d, bool e4m3) {
    SliceDims s;
    s.DH = d.dh <= 64 ? 64 : 128;
    s.ekh = d.rk * (d.d1 + d.d2) + (e4m3 ? 2 : 0);
    s.evh = d.rv * (d.d1 + d.d2) + (e4m3 ? 2 : 0);
    s.ekp = s.ekh | 1;                       // odd stride: the groups' vectors fall in distinct banks
    s.evp = s.evh | 1;
    return s;
}

int smem_bytes(const Dims &d, bool e4m3) {
    const SliceDims s = slice_dims(d, e4m3);
    return layout_of(s.DH, s.ekh, s.evh, s.ekp, s.evp, e4m3).total;
}

// out[row][head] = out_scale * sum_z 2^(m_z - M) o_z / sum_z 2^(m_z - M) l_z over the splits of
// a row; a split that saw nothing (m = -inf, l = 0) is not read.  W warps share a (row, head):
// one when there are few splits or many rows, eight (a whole block) for many splits of few
// rows, so that the loads of a long list run side by side.
template <int W>
__global__ void __launch_bounds__(256) paged_combine_kernel(PagedAttnArgs a, int h, int dh) {
    __shared__ float part[8][128 + 1];                              // features, then l
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long rh = (long long)blockIdx.x * (8 / W) + warp / W;
    if (rh >= (long long)a.n_rows * h) return;
    const int row = (int)(rh / h);
    if (a.cu && (row < a.cu[0] || row >= a.cu[a.batch])) return;    // a row of no sequence
    long long base = rh * a.n_split, stride = 1;
    int n = a.n_split;
    if (a.slots) {
        const int2 s = a.slots[row];
        base = (long long)s.x * h + rh % h, stride = h, n = s.y;
    }
    const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml) + base;
    const float *po = a.part_o + base * dh;
    float M = -INFINITY;
    for (int z = lane; z < n; z += 32) M = fmaxf(M, ml[z * stride].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float l = 0.f;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};                            // features lane + 32 i
    const int z0 = warp % W;
    const float2 *mz = ml + z0 * stride;
    const float *pz = po + z0 * stride * dh + lane;
    const long long step = W * stride;
#pragma unroll 4
    for (int z = z0; z < n; z += W, mz += step, pz += step * dh) {
        const float2 s = *mz;
        if (s.x == -INFINITY && s.y == 0.f) continue;
        const float w = exp2f(s.x - M);
        l += w * s.y;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane + 32 * i < dh) acc[i] += w * pz[32 * i];
    }
    if constexpr (W > 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) part[warp][lane + 32 * i] = acc[i];
        if (lane == 0) part[warp][128] = l;
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int w = 1; w < W; ++w) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] += part[w][lane + 32 * i];
            l += part[w][128];
        }
    }
    const float inv = l == 0.f ? 0.f : a.out_scale / l;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < dh) a.out[rh * dh + lane + 32 * i] = __float2bfloat16_rn(acc[i] * inv);
}

}  // namespace

int paged_mma_rows() { return kRows; }

bool paged_mma_supported(const Dims &d, bool e4m3) {
    if (d.order == 3 || d.shared || d.dh > 128 || d.dh < 2 || d.d2 % 2 != 0) return false;
    return smem_bytes(d, e4m3) <= 226 * 1024;       // (static shared memory beside it)
}

cudaError_t launch_paged_combine(const PagedShape &s, const PagedAttnArgs &a, cudaStream_t st) {
    const long long rh = (long long)a.n_rows * s.d.h;
    const bool wide = a.n_split > 8 && rh < 1024;            // (more rows fill the SMs with a warp each)
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)(wide ? rh : (rh + 7) / 8));
    lc.blockDim = dim3(256);
    lc.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return wide ? cudaLaunchKernelEx(&lc, paged_combine_kernel<8>, a, s.d.h, s.d.dh)
                : cudaLaunchKernelEx(&lc, paged_combine_kernel<1>, a, s.d.h, s.d.dh);
}

namespace {
template <int DH, bool E4M3>
cudaError_t launch_dh(const MmaArgs &a, dim3 grid, size_t smem, cudaStream_t st) {
    cudaError_t e = ensure_dynamic_smem<paged_mma_kernel<DH, E4M3>>(smem);
    if (e != cudaSuccess) return e;
    paged_mma_kernel<DH, E4M3><<<grid, kThreads, smem, st>>>(a);
    return cudaGetLastError();
}
}  // namespace

cudaError_t launch_paged_mma(const PagedShape &s, const PagedAttnArgs &p, cudaStream_t st) {
    const bool e4m3 = s.pool.e4m3 != 0;
    if (!paged_mma_supported(s.d, e4m3)) return cudaErrorInvalidValue;
    const SliceDims sd = slice_dims(s.d, e4m3);
    MmaArgs a;
    a.p = p;
    a.pool = s.pool;
    a.h1 = s.d.h1;
    a.h2 = s.d.h2;
    a.d1 = s.d.d1;
    a.d2 = s.d.d2;
    a.dh = s.d.dh;
    a.rk = s.d.rk;
    a.rv = s.d.rv;
    a.ek = s.d.ek;
    a.ev = s.d.ev;
    a.ekh = sd.ekh;
    a.evh = sd.evh;
    a.ekp = sd.ekp;
    a.evp = sd.evp;
    a.nch = (s.d.d2 + 3) / 4;
    const size_t smem = (size_t)smem_bytes(s.d, e4m3);
    const unsigned tiles = p.cu ? (unsigned)(((long long)p.n_rows + (long long)p.batch * (kRows - 1)) / kRows) : (unsigned)p.batch;
    // (y: at most 65535 row tiles, checked by the caller)
    const dim3 grid((unsigned)s.d.h, tiles, (unsigned)p.n_split);
    cudaError_t e;
    if (sd.DH == 64)
        e = e4m3 ? launch_dh<64, true>(a, grid, smem, st) : launch_dh<64, false>(a, grid, smem, st);
    else
        e = e4m3 ? launch_dh<128, true>(a, grid, smem, st) : launch_dh<128, false>(a, grid, smem, st);
    if (e != cudaSuccess || p.n_split == 1) return e;
    return launch_paged_combine(s, p, st);
}

}  // namespace kpa
