// kpa_paged_write.cu -- records into a paged factor cache and back.
//
// Writing: key B factors are rotated at the token's position (Theorem 2.4 of "Kronecker
// Product Attention"); an e4m3 pool takes each of a token's two parts (A of all ranks, B of
// all ranks) over a power of two, so a code times its scale is exact in bf16 and fp16, and
// the scales of a Kronecker product's two factors multiply into one number per token.
//
// Both directions transpose between token-major records and the pages' element-major
// groups.  One CTA takes one 16-slot group of one plane: the records are read and written
// in order (one warp per token), the group's rows as 16-byte vectors, and the transposition
// goes through shared memory in pieces of kPiece elements, so any record length fits.
// Bound by memory: nothing is read or written twice.
#include "kpa_paged.cuh"

namespace kpa {
namespace {

using namespace paged;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPiece = 512;                       // elements of a record staged at a time

struct WriteArgs {
    Pool pool;
    unsigned char *kpool, *vpool;                 // (append)
    __nv_bfloat16 *kf, *vf;                       // records (append: read only)
    const int32_t *cu, *start;
    int batch, n_rows;
    int ek, ev, ak, av;                           // elements and A elements of a record
    int d2;
    long long max_slots;                          // page_size * table_stride
    int *err;
};

// 16-slot groups that the rows of sequence b touch.
__device__ __forceinline__ long long floor16(long long a) { return a >= 0 ? a / 16 : -((-a + 15) / 16); }

// byte of slot t inside a row of an e4m3 group
__device__ __forceinline__ int byte_of(int t) { return 2 * (t & 7) + (t >> 3); }

struct Group {
    int row0;                                     // row of the group's first token here
    int t0, t1;                                   // its tokens: slots t0 .. t1 - 1 of the group
    long long slot0;                              // first slot of the group
    unsigned char *dst;                           // the group in the pool plane, or null
    bool any;
};

// The group of this CTA: false when there is none.
template <class Plane>
__device__ __forceinline__ bool my_group(const WriteArgs &a, Plane *plane, int bytes, Group &g) {
    const Found f = find_unit<kThreads>(blockIdx.x, a.cu, a.start, a.batch, a.n_rows, a.err, [](long long s, int n) {
        return (int)(floor16(s + n - 1) - floor16(s)) + 1;
    });
    if (f.b < 0) return false;
    const long long s0 = f.pos, n = f.n;
    const long long gi = floor16(s0) + f.i;
    g.slot0 = gi * 16;
    g.t0 = (int)max(0ll, s0 - g.slot0);
    g.t1 = (int)min(16ll, s0 + n - g.slot0);
    g.row0 = f.r0 + (int)(g.slot0 + g.t0 - s0);
    g.dst = nullptr;
    bool ok = g.slot0 >= 0 && g.slot0 + 16 <= a.max_slots;      // (the range is whole groups)
    if (ok) {
        int entry, in;
        split_group(a.pool, (int)gi, entry, in);
        const int page = a.pool.table[(size_t)f.b * a.pool.table_stride + entry];
        ok = page >= 0 && page < a.pool.n_pages;
        if (ok) g.dst = (unsigned char *)plane + ((size_t)page * a.pool.pg + in) * (size_t)bytes;
    }
    if (!ok && threadIdx.x == 0) raise_error(a.err, kErrDeviceCheck);
    return true;
}

// Two neighbouring elements e, e + 1 of a record (e even when VEC: one 4-byte load).
template <bool VEC>
__device__ __forceinline__ float2 load2(const __nv_bfloat16 *r, int e) {
    if constexpr (VEC) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(r + e));
    return make_float2(__bfloat162float(r[e]), __bfloat162float(r[e + 1]));
}

__device__ __forceinline__ float finite_abs(float x) {
    const float y = fabsf(x);
    return y <= 3.4028235e38f ? y : 0.f;          // (false for NaN)
}

// E8M0 byte of a part whose largest finite magnitude is m: the smallest e with 448 2^e >= m.
// 448 = 1.75 * 2^8: adding 0x1fffff to the float's bits carries into the exponent exactly
// when its significand is above 1.75.
__device__ __forceinline__ int scale_byte(float m) {
    const int e = (int)((__float_as_uint(m) + 0x1fffffu) >> 23) - 8;      // biased by 127
    return min(max(e, 63), 190);
}

template <bool E4M3, bool VEC>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(WriteArgs a, RopeTable rope) {
    // e4m3: [kPiece][16] codes; bf16: [2][kPiece][8]
    __shared__ __align__(16) unsigned char tile[kPiece * (E4M3 ? 16 : 32)];
    __shared__ float2 cs[16][kMaxHalfD2 + 1];
    __shared__ uint32_t scales[16];               // exponent bytes: A in the low byte, B in the next
    const bool is_k = blockIdx.y == 0;
    const int E = is_k ? a.ek : a.ev, A = is_k ? a.ak : a.av;
    Group g;
    if (!my_group(a, is_k ? a.kpool : a.vpool, is_k ? a.pool.kg : a.pool.vg, g) || !g.dst) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int half = a.d2 / 2;
    if (is_k) {
        for (int i = tid; i < (g.t1 - g.t0) * half; i += kThreads) {
            const int t = g.t0 + i / half, m = i % half;
            float c, s;
            rope_cs((double)(g.slot0 + t), rope.theta[m], c, s);
            cs[t][m] = make_float2(c, s);
        }
        __syncthreads();
    }
    const __nv_bfloat16 *src = is_k ? a.kf : a.vf;
    // Elements 2p, 2p + 1 counted over A then B, each part rounded up to whole pairs; the
    // second element of an odd A part's last pair is absent (dropped by every user).
    const int pa = (A + 1) / 2, pairs = pa + (E - A) / 2;
    auto pair_at = [&](const __nv_bfloat16 *r, int t, int p, int &e, bool &one) -> float2 {
        const bool in_b = p >= pa;
        e = in_b ? A + 2 * (p - pa) : 2 * p;
        one = !in_b && e + 1 >= A;
        if (one) return make_float2(__bfloat162float(r[e]), 0.f);
        float2 x = load2<VEC>(r, e);
        if (in_b && is_k) {
            const float2 w = cs[t][(p - pa) % half];
            x = make_float2(x.x * w.x - x.y * w.y, x.x * w.y + x.y * w.x);
        }
        return x;
    };
    if constexpr (E4M3) {
        for (int t = g.t0 + warp; t < g.t1; t += kWarps) {
            const __nv_bfloat16 *r = src + (size_t)(g.row0 + t - g.t0) * E;
            float ma = 0.f, mb = 0.f;
            for (int p = lane; p < pairs; p += 32) {
                int e;
                bool one;
                const float2 x = pair_at(r, t, p, e, one);
                const float m = fmaxf(finite_abs(x.x), finite_abs(x.y));
                if (p >= pa)
                    mb = fmaxf(mb, m);
                else
                    ma = fmaxf(ma, m);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, off));
                mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, off));
            }
            if (lane == 0) scales[t] = (uint32_t)scale_byte(ma) | ((uint32_t)scale_byte(mb) << 8);
        }
        __syncthreads();
        // the scale rows
        if (tid >= g.t0 && tid < g.t1) {
            g.dst[(size_t)E * 16 + byte_of(tid)] = (unsigned char)(scales[tid] & 255u);
            g.dst[(size_t)(E + 1) * 16 + byte_of(tid)] = (unsigned char)(scales[tid] >> 8);
        }
    }
    const bool full = g.t0 == 0 && g.t1 == 16;
    for (int p0 = 0; p0 < pairs; p0 += kPiece / 2) {
        const int p1 = min(p0 + kPiece / 2, pairs);
        // elements [e0, e1) of this piece
        auto elem = [&](int p) { return p >= pa ? A + 2 * (p - pa) : 2 * p; };
        const int e0 = elem(p0), e1 = p1 == pairs ? E : elem(p1);
        if (p0) __syncthreads();
        for (int t = g.t0 + warp; t < g.t1; t += kWarps) {
            const __nv_bfloat16 *r = src + (size_t)(g.row0 + t - g.t0) * E;
            float sa = 1.f, sb = 1.f;
            if constexpr (E4M3) {                 // 2^-e, e = byte - 127 in [-64, 63]
                sa = exp_byte(254u - (scales[t] & 255u));
                sb = exp_byte(254u - (scales[t] >> 8));
            }
            for (int p = p0 + lane; p < p1; p += 32) {
                int e;
                bool one;
                float2 x = pair_at(r, t, p, e, one);
                if constexpr (E4M3) {
                    const float s = p >= pa ? sb : sa;
                    // infinities become NaN (the conversion would saturate them)
                    x.x = fabsf(x.x) <= 3.4028235e38f ? x.x * s : __uint_as_float(0x7fffffffu);
                    x.y = fabsf(x.y) <= 3.4028235e38f ? x.y * s : __uint_as_float(0x7fffffffu);
                    const uint32_t c = to_e4m3x2(x.x, x.y);
                    tile[(e - e0) * 16 + byte_of(t)] = (unsigned char)(c & 255u);
                    if (!one) tile[(e + 1 - e0) * 16 + byte_of(t)] = (unsigned char)(c >> 8);
                } else {
                    __nv_bfloat16 *tb = reinterpret_cast<__nv_bfloat16 *>(tile) + (t >> 3) * (kPiece * 8);
                    tb[(e - e0) * 8 + (t & 7)] = __float2bfloat16_rn(x.x);
                    if (!one) tb[(e + 1 - e0) * 8 + (t & 7)] = __float2bfloat16_rn(x.y);
                }
            }
        }
        __syncthreads();
        const int n = e1 - e0;
        if constexpr (E4M3) {
            unsigned char *dst = g.dst + (size_t)e0 * 16;
            if (full) {
                for (int i = tid; i < n; i += kThreads)
                    reinterpret_cast<uint4 *>(dst)[i] = reinterpret_cast<const uint4 *>(tile)[i];
            } else {
                const int nt = g.t1 - g.t0;
                for (int i = tid; i < n * nt; i += kThreads) {
                    const int e = i / nt, o = e * 16 + byte_of(g.t0 + i % nt);
                    dst[o] = tile[o];
                }
            }
        } else {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int lo = max(g.t0 - 8 * hf, 0), hi = min(g.t1 - 8 * hf, 8);
                if (lo >= hi) continue;
                __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(g.dst) + ((size_t)hf * E + e0) * 8;
                const __nv_bfloat16 *tb = reinterpret_cast<const __nv_bfloat16 *>(tile) + hf * (kPiece * 8);
                if (hi - lo == 8) {
                    for (int i = tid; i < n; i += kThreads)
                        reinterpret_cast<uint4 *>(dst)[i] = reinterpret_cast<const uint4 *>(tb)[i];
                } else {
                    for (int i = tid; i < n * (hi - lo); i += kThreads) {
                        const int o = (i / (hi - lo)) * 8 + lo + i % (hi - lo);
                        dst[o] = tb[o];
                    }
                }
            }
        }
    }
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads) paged_read_kernel(WriteArgs a) {
    __shared__ __align__(16) unsigned char tile[kPiece * (E4M3 ? 16 : 32)];
    __shared__ __align__(16) unsigned char sc[32];
    const bool is_k = blockIdx.y == 0;
    const int E = is_k ? a.ek : a.ev, A = is_k ? a.ak : a.av;
    Group g;
    if (!my_group(a, is_k ? a.pool.k : a.pool.v, is_k ? a.pool.kg : a.pool.vg, g)) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __nv_bfloat16 *rec = is_k ? a.kf : a.vf;
    if (!g.dst) {
        for (long long i = tid; i < (long long)(g.t1 - g.t0) * E; i += kThreads)
            rec[(size_t)g.row0 * E + i] = __float2bfloat16_rn(0.f);
        return;
    }
    if constexpr (E4M3) {
        if (tid < 2) reinterpret_cast<uint4 *>(sc)[tid] = reinterpret_cast<const uint4 *>(g.dst)[E + tid];
    }
    for (int e0 = 0; e0 < E; e0 += kPiece) {
        const int n = min(kPiece, E - e0);
        if (e0) __syncthreads();
        if constexpr (E4M3) {
            for (int i = tid; i < n; i += kThreads)
                reinterpret_cast<uint4 *>(tile)[i] = reinterpret_cast<const uint4 *>(g.dst)[e0 + i];
        } else {
            for (int i = tid; i < 2 * n; i += kThreads) {
                const int hf = i >= n, e = hf ? i - n : i;
                reinterpret_cast<uint4 *>(tile)[hf * kPiece + e] =
                    reinterpret_cast<const uint4 *>(g.dst)[(size_t)hf * E + e0 + e];
            }
        }
        __syncthreads();
        for (int t = g.t0 + warp; t < g.t1; t += kWarps) {
            __nv_bfloat16 *r = rec + (size_t)(g.row0 + t - g.t0) * E + e0;
            for (int e = lane; e < n; e += 32) {
                if constexpr (E4M3) {
                    const float s = exp_byte(sc[(e0 + e >= A ? 16 : 0) + byte_of(t)]);
                    const float2 f = h2_to_f2(e4m3x2_to_h2(tile[e * 16 + byte_of(t)]));
                    r[e] = __float2bfloat16_rn(f.x * s);
                } else {
                    r[e] = reinterpret_cast<const __nv_bfloat16 *>(tile)[((t >> 3) * kPiece + e) * 8 + (t & 7)];
                }
            }
        }
    }
}

WriteArgs write_args(const PagedShape &s, int batch, int n_rows, const int32_t *cu, const int32_t *start, int *err) {
    WriteArgs a = {};
    a.pool = s.pool;
    a.cu = cu;
    a.start = start;
    a.batch = batch;
    a.n_rows = n_rows;
    a.ek = s.d.ek;
    a.ev = s.d.ev;
    a.ak = s.d.rk * s.d.h1 * s.d.d1;
    a.av = s.d.rv * s.d.h1 * s.d.d1;
    a.d2 = s.d.d2;
    a.max_slots = (long long)s.pool.pg * 16 * s.pool.table_stride;
    a.err = err;
    return a;
}

// n rows of one sequence touch at most (n + 14) / 16 + 1 groups
dim3 write_grid(int batch, int n_rows) {
    return dim3((unsigned)(((long long)n_rows + 14ll * batch) / 16 + batch), 2);
}

}  // namespace

cudaError_t launch_paged_append(const PagedShape &s, int batch, int n_rows, const void *kf, const void *vf,
                                const int32_t *cu, const int32_t *start, void *kpool, void *vpool,
                                const RopeTable &rope, int *err, cudaStream_t st) {
    WriteArgs a = write_args(s, batch, n_rows, cu, start, err);
    a.kf = const_cast<__nv_bfloat16 *>(static_cast<const __nv_bfloat16 *>(kf));
    a.vf = const_cast<__nv_bfloat16 *>(static_cast<const __nv_bfloat16 *>(vf));
    a.kpool = static_cast<unsigned char *>(kpool);
    a.vpool = static_cast<unsigned char *>(vpool);
    const dim3 grid = write_grid(batch, n_rows);
    // pairs of records and of their B parts start on 4-byte boundaries
    const bool vec = a.ek % 2 == 0 && a.ev % 2 == 0 && a.ak % 2 == 0 && a.av % 2 == 0;
    if (s.pool.e4m3) {
        if (vec)
            paged_append_kernel<true, true><<<grid, kThreads, 0, st>>>(a, rope);
        else
            paged_append_kernel<true, false><<<grid, kThreads, 0, st>>>(a, rope);
    } else {
        if (vec)
            paged_append_kernel<false, true><<<grid, kThreads, 0, st>>>(a, rope);
        else
            paged_append_kernel<false, false><<<grid, kThreads, 0, st>>>(a, rope);
    }
    return cudaGetLastError();
}

cudaError_t launch_paged_read(const PagedShape &s, int batch, int n_rows, const int32_t *cu, const int32_t *start,
                              void *kf, void *vf, int *err, cudaStream_t st) {
    WriteArgs a = write_args(s, batch, n_rows, cu, start, err);
    a.kf = static_cast<__nv_bfloat16 *>(kf);
    a.vf = static_cast<__nv_bfloat16 *>(vf);
    const dim3 grid = write_grid(batch, n_rows);
    if (s.pool.e4m3)
        paged_read_kernel<true><<<grid, kThreads, 0, st>>>(a);
    else
        paged_read_kernel<false><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace kpa
