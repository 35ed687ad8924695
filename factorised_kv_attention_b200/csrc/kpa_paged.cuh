// kpa_paged.cuh -- the paged factor cache as the kernels see it: where a slot lies, which
// slots a row sees, and which rows belong to which sequence.
#pragma once

#include "kpa_internal.cuh"

namespace kpa {
namespace paged {

constexpr int kSlots16 = 16;         // slots per addressed group (two 8-slot groups in a bf16 page)

// One pool and its page table.  Both formats are addressed by groups of 16 slots: a group
// of a plane is one contiguous run of kg (vg) bytes, E * 32 in bf16, (E + 2) * 16 in e4m3.
struct Pool {
    const unsigned char *k, *v;
    const int32_t *table;
    int table_stride;
    int n_pages;
    int pg;                          // groups per page
    unsigned long long magic;        // ceil(2^36 / pg): group / pg = group * magic >> 36 for group < 2^27, pg <= 2^8
    int kg, vg;                      // bytes per group of a plane
    int e4m3;
};

// Page table entry index and group inside the page of 16-slot group g of a sequence.
__device__ __forceinline__ void split_group(const Pool &p, int g, int &entry, int &in) {
    entry = (int)(((unsigned long long)(unsigned)g * p.magic) >> 36);
    in = g - entry * p.pg;
}

// Which slots a row at position pos sees: every one up to pos without a window, else [0, sinks)
// and [pos - window + 1, pos].
struct Mask {
    int window, sinks;
};
__host__ __device__ __forceinline__ int window_start(const Mask &m, int pos) {
    return m.window > 0 && pos >= m.window ? pos - m.window + 1 : 0;
}
__device__ __forceinline__ bool sees(const Mask &m, int pos, int s) {
    return s <= pos && (m.window == 0 || pos - s < m.window || s < m.sinks);
}

// The tiles (T slots each, aligned to T) that rows at positions lo .. hi see between them:
// tiles [0, head) hold the sinks and [first, last] the windows; tile v of n is v or v + gap.
struct Tiles {
    int head, gap, n;
    __device__ __forceinline__ int slot_tile(int v) const { return v < head ? v : v + gap; }
};
__device__ __forceinline__ Tiles visible_tiles(const Mask &m, int lo, int hi, int T) {
    Tiles t;
    const int first = window_start(m, lo) / T, last = hi / T;
    const int sink_slots = m.window > 0 ? min(m.sinks, hi + 1) : 0;
    const int sink_tiles = sink_slots > 0 ? (sink_slots - 1) / T + 1 : 0;        // (sinks up to INT_MAX)
    t.head = min(sink_tiles, first);
    t.gap = first - t.head;
    t.n = t.head + (last - first + 1);
    return t;
}

// Run `split` of n tiles cut into n_split runs that differ by at most one tile: [v0, v1).
__device__ __forceinline__ void split_run(int n, int split, int n_split, int &v0, int &v1) {
    v0 = 0, v1 = n;
    if (n_split > 1) {
        const int q = (int)((unsigned)n / (unsigned)n_split), r = n - q * n_split;
        v0 = split * q + min(split, r);
        v1 = v0 + q + (split < r ? 1 : 0);
    }
}

// Finds the sequence that unit `idx` falls to when a sequence of n rows from position p has
// count(p, n) units, laid one sequence after the other: its rows r0 .. r0 + n - 1, its first
// position and the unit's index i inside it (b = -1 past the last unit).  Every thread of the
// block calls it (whole warps, at most 32); each step scans as many sequences as the block has
// threads, to the end of the batch in the block that reports sequences with rows outside
// [0, n_rows].
struct Found {
    int b, i, r0, n, pos;
};
template <class Count>
__device__ __forceinline__ Found find_unit(int idx, const int32_t *cu, const int32_t *start, int batch, int n_rows,
                                           int *err, Count count) {
    __shared__ int warp_sum[32];
    __shared__ Found hit;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
    if (tid == 0) hit.b = -1;
    int before = 0;
    for (int base = 0; base < batch; base += threads) {
        const int b = base + tid;
        int c = 0;
        Found f = {b, 0, 0, 0, 0};
        if (b < batch) {
            f.r0 = cu[b];
            const int r1 = cu[b + 1];
            f.pos = start[b];
            if (f.r0 < 0 || r1 < f.r0 || r1 > n_rows) {
                if (idx == 0) raise_error(err, kErrDeviceCheck);
            } else {
                f.n = r1 - f.r0;
                c = f.n > 0 ? count(f.pos, f.n) : 0;
            }
        }
        int inc = c;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += v;
        }
        if (lane == 31) warp_sum[warp] = inc;
        __syncthreads();
        int pre = before, total = before;
        for (int w = 0; w < threads / 32; ++w) {
            const int s = warp_sum[w];
            if (w < warp) pre += s;
            total += s;
        }
        const int lo = pre + inc - c;
        if (idx >= lo && idx < lo + c) {
            f.i = idx - lo;
            hit = f;
        }
        __syncthreads();
        before = total;
        if (idx != 0 && idx < before) break;
    }
    return hit;
}

// The same for row tiles of T rows in the order of what they cost: level 0 holds the last
// tile of every sequence, level 1 the one before it, and so on, sequences in order within a
// level, so that long rows start first and the last blocks are short.  i is the tile's index
// from the sequence's front.  With ShortLast a sequence's last tile comes after all of these where
// it holds at most T / 2 rows (it costs about half there).  (Batches above 256 sequences:
// sequence after sequence, its last tile first.)
template <int T, bool ShortLast = false>
__device__ __forceinline__ Found find_tile(int idx, const int32_t *cu, const int32_t *start, int batch, int n_rows,
                                           int *err) {
    if (batch > 256) {
        Found f = find_unit(idx, cu, start, batch, n_rows, err, [](int, int n) { return (n + T - 1) / T; });
        if (f.b >= 0) f.i = (f.n + T - 1) / T - 1 - f.i;
        return f;
    }
    __shared__ Found hit;
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        // a sequence's tiles in the levels: all, or with ShortLast all but a short last one
        auto levels = [](int n) { return ShortLast ? (n + (T - T / 2 - 1)) / T : (n + T - 1) / T; };
        int n[8], r0[8], pos[8], most = 0, all = 0;                 // sequences lane + 32 k
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int b = lane + 32 * k;
            n[k] = r0[k] = pos[k] = 0;
            if (b < batch) {
                r0[k] = cu[b];
                const int r1 = cu[b + 1];
                pos[k] = start[b];
                if (r0[k] < 0 || r1 < r0[k] || r1 > n_rows) {
                    if (idx == 0) raise_error(err, kErrDeviceCheck);
                } else {
                    n[k] = r1 - r0[k];
                }
            }
            most = max(most, levels(n[k]));
            all += levels(n[k]);
        }
        most = (int)__reduce_max_sync(0xffffffffu, (unsigned)most);
        all = (int)__reduce_add_sync(0xffffffffu, (unsigned)all);
        if (lane == 0) hit.b = -1;
        __syncwarp();
        const bool in_levels = idx < all;
        // the largest level whose first unit is no later than idx; before: units of the levels below
        int lo = 0, hi = in_levels ? most : 0, before = in_levels ? 0 : all;       // lo is one, hi is not
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            int c = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) c += min(levels(n[k]), mid);
            c = (int)__reduce_add_sync(0xffffffffu, (unsigned)c);
            if (c <= idx) {
                lo = mid;
                before = c;
            } else {
                hi = mid;
            }
        }
        int rank = idx - before;                                    // among the sequences that reach the level
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int t = levels(n[k]);
            const bool has = in_levels ? t > lo : (n[k] + T - 1) / T > t;          // (past the levels: a short tile)
            const unsigned m = __ballot_sync(0xffffffffu, has);
            if (has && rank >= 0 && __popc(m & ((1u << lane) - 1u)) == rank) {
                hit.b = lane + 32 * k;
                hit.i = in_levels ? t - 1 - lo : t;
                hit.r0 = r0[k];
                hit.n = n[k];
                hit.pos = pos[k];
            }
            rank -= __popc(m);                                      // (negative once found)
        }
    }
    __syncthreads();
    return hit;
}

// ---- e4m3
// two e4m3 codes (low byte first) as fp16x2
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
// (lo, hi) floats as two e4m3 codes, nearest even, saturating at 448; NaN stays NaN
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e4m3x2.f32 c, %1, %2;\n\tcvt.u32.u16 %0, c;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 h2_to_f2(uint32_t w) {
    float2 f;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(w));
    return f;
}
// Four e4m3 bytes of a group row or column pair, in the order slot, slot + 8 of one value,
// then of the next: the two values of the lower slots and of the upper slots, as fp16x2.
__device__ __forceinline__ void e4m3_split(uint32_t w, uint32_t &lower, uint32_t &upper) {
    const uint32_t v = __byte_perm(w, 0, 0x3120);
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lower), "=r"(upper)
        : "r"(v));
}
// 2^(byte - 127) for byte in [1, 254]
__device__ __forceinline__ float exp_byte(uint32_t byte) { return __uint_as_float(byte << 23); }
// Four slots' exponent bytes of the A row and of the B row (each in [63, 190] for a slot that
// was written) to the bytes of their products' exponents: 2^(a - 127) 2^(b - 127) =
// 2^((a + b - 126) - 128), a + b - 126 in [0, 254].  Each byte's sum is taken modulo 256
// without a carry into its neighbour: an unwritten slot beside may hold anything.
__device__ __forceinline__ uint32_t exp_sum4(uint32_t a4, uint32_t b4) {
    const uint32_t t = ((a4 & 0x7f7f7f7fu) + (b4 & 0x7f7f7f7fu)) ^ ((a4 ^ b4) & 0x80808080u);
    return ((t & 0x7f7f7f7fu) + 0x02020202u) ^ (~t & 0x80808080u);          // + 130 = - 126
}
// 2^(byte - 128), byte in [1, 254]: half of 2^(byte - 127).  0 for byte 0, where both exponents are
// the smallest that are written, -64: products below 2^-110.
__device__ __forceinline__ float exp_sum(uint32_t byte) { return 0.5f * __uint_as_float(byte << 23); }

}  // namespace paged

// ---- host-side launchers
struct PagedShape {
    Dims d;
    paged::Pool pool;
};

cudaError_t launch_paged_append(const PagedShape &s, int batch, int n_rows, const void *kf, const void *vf,
                                const int32_t *cu, const int32_t *start, void *kpool, void *vpool,
                                const RopeTable &rope, int *err, cudaStream_t st);
cudaError_t launch_paged_read(const PagedShape &s, int batch, int n_rows, const int32_t *cu, const int32_t *start,
                              void *kf, void *vf, int *err, cudaStream_t st);

// Attention of rows (cu, start) or, with cu null, of one row per sequence at position
// seq_len[b] - 1.
struct PagedAttnArgs {
    const __nv_bfloat16 *q;
    const int32_t *cu, *start, *seq_len;
    int batch, n_rows, max_len;
    paged::Mask mask;
    float qscale;                 // sm_scale / R_K * log2(e)
    float out_scale;              // 1 / R_V
    __nv_bfloat16 *out;
    float *part_o, *part_ml;      // n_split > 1: [n_rows][h][n_split][d_h] and [n_rows][h][n_split][2]
    int n_split;
    int2 *slots;                  // splits sized on the device: (first slot, slots) of each sequence, and the
                                  // partials are [slot][h][d_h] and [slot][h][2]; else null
    int *err;
};

bool paged_mma_supported(const Dims &d, bool e4m3);
int paged_mma_rows();                                        // rows of a tile
cudaError_t launch_paged_mma(const PagedShape &s, const PagedAttnArgs &a, cudaStream_t st);
cudaError_t launch_paged_combine(const PagedShape &s, const PagedAttnArgs &a, cudaStream_t st);

// The tcgen05 chunk kernel: whether it takes this shape and pool, and its launcher.
bool paged_prefill_supported(const PagedShape &s);
int paged_prefill_rows();                                    // rows of a tile
cudaError_t launch_paged_prefill(const PagedShape &s, const PagedAttnArgs &a, unsigned long long wait_limit_ns,
                                 cudaStream_t st);

// The single-token kernel: its variant for these dims (-1: none, the chunk kernel takes
// them), the 16-slot groups of its tiles and its CTAs per SM, and its launcher.
int paged_decode_variant(const Dims &d);
void paged_decode_shape(int variant, bool e4m3, int *tile_groups, int *ctas_per_sm);
constexpr int kPagedMaxCluster = 16;
int paged_decode_max_clusters(int variant, bool e4m3, int size);     // resident at once (at least 2 CTAs each)
// groups_per_split: of a grid of n_split x batch blocks; with a.slots, n_slots blocks size the
// splits themselves.
cudaError_t launch_paged_decode(int variant, const PagedShape &s, const PagedAttnArgs &a, int groups_per_split,
                                int n_slots, bool cluster, unsigned long long wait_limit_ns, cudaStream_t st);
constexpr int kPagedMaxSlotSeqs = 256;                       // sequences that such a block can place

}  // namespace kpa
