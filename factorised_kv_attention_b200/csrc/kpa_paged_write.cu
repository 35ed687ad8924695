// kpa_paged_write.cu -- records into a paged factor cache and back.
//
// Writing: key B factors are rotated at the token's position (Theorem 2.4 of "Kronecker
// Product Attention"); an e4m3 pool takes each of a token's two parts (A of all ranks, B of
// all ranks) over a power of two, so a code times its scale is exact in bf16 and fp16, and
// the scales of a Kronecker product's two factors multiply into one number per token.
//
// Both directions transpose between token-major records and the pages' element-major
// groups.  One CTA takes one 16-slot group of one plane, one thread two neighbouring elements
// of all 16 slots: a warp reads (writes) 128 contiguous bytes of each record and writes
// (reads) whole 16-byte rows of the group, and the transposition is the thread's registers.
// Nothing goes through shared memory but the rotation table and the largest magnitudes of
// the 16 tokens.  Bound by latency at a few tokens (4.4 us for 48) and by issue slots beyond:
// 16384 tokens of 384 values written as e4m3 in 12.0 us (1.6 TB/s; 66 % of the issue slots), 16384
// of 576 read back in 9.5 us (3.0 TB/s).
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "kpa_paged.cuh"

namespace kpa {
namespace {

using namespace paged;


constexpr int kMaxThreads = 512;

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

// a / 16 rounded down, positions below 0 too
__device__ __forceinline__ long long floor16(long long a) { return a >= 0 ? a / 16 : -((-a + 15) / 16); }

// byte of slot t inside a row of an e4m3 group
__device__ __forceinline__ int byte_of(int t) { return 2 * (t & 7) + (t >> 3); }

struct Group {
    int b;                                        // its sequence
    int row0;                                     // row of the group's first token here
    int t0, t1;                                   // its tokens: slots t0 .. t1 - 1 of the group
    long long slot0;                              // first slot of the group
};

// The group of this CTA: false when there is none.
__device__ __forceinline__ bool find_group(const WriteArgs &a, Group &g) {
    const Found f = find_unit(blockIdx.x, a.cu, a.start, a.batch, a.n_rows, a.err, [](long long s, int n) {
        return (int)(floor16(s + n - 1) - floor16(s)) + 1;
    });
    if (f.b < 0) return false;
    const long long s0 = f.pos, n = f.n;
    g.b = f.b;
    g.slot0 = (floor16(s0) + f.i) * 16;
    g.t0 = (int)max(0ll, s0 - g.slot0);
    g.t1 = (int)min(16ll, s0 + n - g.slot0);
    g.row0 = f.r0 + (int)(g.slot0 + g.t0 - s0);
    return true;
}

// Which group of the pool it is, or -1: reported.
__device__ __forceinline__ long long pool_group(const WriteArgs &a, const Group &g) {
    if (g.slot0 >= 0 && g.slot0 + 16 <= a.max_slots) {          // (the table's range is whole groups)
        int entry, in;
        split_group(a.pool, (int)(g.slot0 >> 4), entry, in);
        const int page = __ldg(a.pool.table + (size_t)g.b * a.pool.table_stride + entry);
        if (page >= 0 && page < a.pool.n_pages) return (long long)page * a.pool.pg + in;
    }
    if (threadIdx.x == 0) raise_error(a.err, kErrDeviceCheck);
    return -1;
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

// Largest of each of 16 values over the warp: lane l returns that of value
// 8 l[4] + 4 l[3] + 2 l[2] + l[1] (bits of l).  Each step trades half of the values.
__device__ __forceinline__ float warp_max16(float (&v)[16], int lane) {
#pragma unroll
    for (int n = 8; n >= 1; n >>= 1) {
        const bool up = lane & (2 * n);
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
            v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 2 * n));
        }
    }
    return fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

// VEC: records, and their B parts, start on 4-byte boundaries (two elements per load).
template <bool E4M3, bool VEC>
__global__ void __launch_bounds__(kMaxThreads, 2) paged_append_kernel(WriteArgs a, RopeTable rope) {
    extern __shared__ float2 cs[];                // [d2 / 2][16]: (cos, sin) of pair m at slot t
    __shared__ unsigned top[2][16];               // bits of the parts' largest magnitudes
    const bool is_k = blockIdx.y == 0;
    const int E = is_k ? a.ek : a.ev, A = is_k ? a.ak : a.av;
    const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x;
    if (tid < 32) top[tid >> 4][tid & 15] = 0u;   // (the scan below synchronises)
    Group g;
    if (!find_group(a, g)) return;
    const int half = a.d2 / 2;
    // Pair p is elements 2p, 2p + 1 of A, then of B; the last pair of an odd A has one.
    const int pa = (A + 1) / 2, pairs = pa + (E - A) / 2;
    const __nv_bfloat16 *src = (is_k ? a.kf : a.vf) + (size_t)g.row0 * E - (size_t)g.t0 * E;
    uint32_t x[16];
    auto load = [&](int p) {
        const int e = p >= pa ? A + 2 * (p - pa) : 2 * p;
        const bool one = p < pa && e + 1 >= A;
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            x[t] = 0u;
            if (p < pairs && t >= g.t0 && t < g.t1) {
                const __nv_bfloat16 *r = src + (size_t)t * E + e;
                if (VEC)
                    x[t] = __ldg(reinterpret_cast<const uint32_t *>(r));
                else
                    x[t] = (uint32_t)__bfloat16_as_ushort(r[0]) | (one ? 0u : (uint32_t)__bfloat16_as_ushort(r[1]) << 16);
            }
        }
    };
    float2 v[16];                                 // the pair's values, rotated for a key's B
    auto rotate = [&](int p) {
        const bool turn = is_k && p >= pa && p < pairs;
        const float2 *w = cs + (turn ? ((p - pa) % half) * 16 : 0);
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            v[t] = make_float2(__uint_as_float(x[t] << 16), __uint_as_float(x[t] & 0xffff0000u));
            if (turn) v[t] = make_float2(v[t].x * w[t].x - v[t].y * w[t].y, v[t].x * w[t].y + v[t].y * w[t].x);
        }
    };
    load(tid);                                    // in flight while the table entry and the angles are
    const long long at = pool_group(a, g);
    if (at < 0) return;
    unsigned char *const dst0 = is_k ? a.kpool + (size_t)at * a.pool.kg : a.vpool + (size_t)at * a.pool.vg;
    if (is_k) {
        for (int i = tid; i < 16 * half; i += threads) {
            const int t = i & 15;
            float c = 0.f, s = 0.f;               // (the rotation of an absent slot's zeros)
            if (t >= g.t0 && t < g.t1) rope_cs((double)(g.slot0 + t), rope.theta[i >> 4], c, s);
            cs[i] = make_float2(c, s);
        }
        __syncthreads();
    }
    rotate(tid);
    const bool once = pairs <= threads;           // the values stay in registers
    if constexpr (E4M3) {
        const int token = ((lane >> 4) & 1) * 8 + ((lane >> 3) & 1) * 4 + ((lane >> 2) & 1) * 2 + ((lane >> 1) & 1);
        for (int p0 = 0; p0 < pairs; p0 += threads) {
            const int p = p0 + tid;
            if (p0) {
                load(p);
                rotate(p);
            }
            const bool in_b = p >= pa;
#pragma unroll 1
            for (int part = 0; part < 2; ++part) {
                if (!__any_sync(0xffffffffu, in_b == (part == 1))) continue;
                float w[16];
#pragma unroll
                for (int t = 0; t < 16; ++t) w[t] = in_b == (part == 1) ? fmaxf(finite_abs(v[t].x), finite_abs(v[t].y)) : 0.f;
                const float mx = warp_max16(w, lane);
                if (!(lane & 1)) atomicMax(&top[part][token], __float_as_uint(mx));   // magnitudes: ordered as bits
            }
        }
        __syncthreads();
        if (tid < 32) {                           // the two scale rows
            const int part = tid >> 4, t = tid & 15;
            if (t >= g.t0 && t < g.t1)
                dst0[(size_t)(E + part) * 16 + byte_of(t)] = (unsigned char)scale_byte(__uint_as_float(top[part][t]));
        }
    }
    const bool full = g.t0 == 0 && g.t1 == 16;
    for (int p0 = 0; p0 < pairs; p0 += threads) {
        const int p = p0 + tid;
        if (!once) {
            load(p);
            rotate(p);
        }
        if (p >= pairs) break;
        const int e = p >= pa ? A + 2 * (p - pa) : 2 * p;
        const bool one = p < pa && e + 1 >= A;
        if constexpr (E4M3) {
            uint32_t w0[4] = {0, 0, 0, 0}, w1[4] = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < 8; ++k) {         // slots k and k + 8: neighbouring bytes
                float2 y[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int t = k + 8 * u;
                    // 2^-e, e = byte - 127 in [-64, 63]
                    const float s = exp_byte(254u - (uint32_t)scale_byte(__uint_as_float(top[p >= pa][t])));
                    // infinities become NaN (the conversion would saturate them)
                    y[u].x = fabsf(v[t].x) <= 3.4028235e38f ? v[t].x * s : __uint_as_float(0x7fffffffu);
                    y[u].y = fabsf(v[t].y) <= 3.4028235e38f ? v[t].y * s : __uint_as_float(0x7fffffffu);
                }
                w0[k >> 1] |= to_e4m3x2(y[0].x, y[1].x) << (16 * (k & 1));
                w1[k >> 1] |= to_e4m3x2(y[0].y, y[1].y) << (16 * (k & 1));
            }
            unsigned char *dst = dst0 + (size_t)e * 16;
            if (full) {
                reinterpret_cast<uint4 *>(dst)[0] = make_uint4(w0[0], w0[1], w0[2], w0[3]);
                if (!one) reinterpret_cast<uint4 *>(dst)[1] = make_uint4(w1[0], w1[1], w1[2], w1[3]);
            } else {
#pragma unroll
                for (int t = 0; t < 16; ++t)
                    if (t >= g.t0 && t < g.t1) {
                        const int o = byte_of(t);
                        dst[o] = (unsigned char)(w0[o >> 2] >> (8 * (o & 3)));
                        if (!one) dst[16 + o] = (unsigned char)(w1[o >> 2] >> (8 * (o & 3)));
                    }
            }
        } else {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                __nv_bfloat16 r0[8], r1[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    r0[k] = __float2bfloat16_rn(v[8 * hf + k].x);
                    r1[k] = __float2bfloat16_rn(v[8 * hf + k].y);
                }
                __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(dst0) + ((size_t)hf * E + e) * 8;
                if (g.t0 <= 8 * hf && g.t1 >= 8 * hf + 8) {
                    uint4 u0, u1;
                    memcpy(&u0, r0, 16);
                    memcpy(&u1, r1, 16);
                    reinterpret_cast<uint4 *>(dst)[0] = u0;
                    if (!one) reinterpret_cast<uint4 *>(dst)[1] = u1;
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (8 * hf + k >= g.t0 && 8 * hf + k < g.t1) {
                            dst[k] = r0[k];
                            if (!one) dst[8 + k] = r1[k];
                        }
                }
            }
        }
    }
}

// VEC: records start on 4-byte boundaries.  One CTA takes a group's keys and values, whose loads
// are in flight together.
template <bool E4M3, bool VEC>
__global__ void __launch_bounds__(kMaxThreads, 2) paged_read_kernel(WriteArgs a) {
    Group g;
    if (!find_group(a, g)) return;
    const long long at = pool_group(a, g);
    const int tid = threadIdx.x, threads = blockDim.x;
    constexpr int N = E4M3 ? 1 : 2;               // 16-byte vectors of an element's 16 slots
    struct Plane {
        const uint4 *rows;                        // the group's, or null (zeros are read)
        int E, A;
        __nv_bfloat16 *rec;                       // of slot 0 of the group
    };
    auto plane = [&](bool is_k) {
        Plane p;
        p.E = is_k ? a.ek : a.ev;
        p.A = is_k ? a.ak : a.av;
        p.rows = at < 0 ? nullptr
                        : reinterpret_cast<const uint4 *>(is_k ? a.pool.k + (size_t)at * a.pool.kg : a.pool.v + (size_t)at * a.pool.vg);
        p.rec = (is_k ? a.kf : a.vf) + ((long long)g.row0 - g.t0) * p.E;
        return p;
    };
    // elements e, e + 1 (the last of an odd record has no second) and the scale row of e's part
    auto load = [&](const Plane &p, int e, uint4 (&x)[2][N], uint4 &scale) {
        if (E4M3) scale = p.rows && e < p.E ? __ldg(p.rows + p.E + (e < p.A ? 0 : 1)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < N; ++n)
                x[i][n] = p.rows && e + i < p.E ? __ldg(p.rows + (size_t)n * p.E + e + i) : make_uint4(0, 0, 0, 0);
    };
    auto emit = [&](const Plane &p, int e, const uint4 (&x)[2][N], const uint4 s0) {
        if (e >= p.E) return;
        uint32_t w[16];                           // the pair at each slot
        if constexpr (E4M3) {
            const uint4 s1 = p.rows && e + 1 == p.A ? __ldg(p.rows + p.E + 1) : s0;      // (an odd A ends between them)
            const uint32_t c0[4] = {x[0][0].x, x[0][0].y, x[0][0].z, x[0][0].w}, c1[4] = {x[1][0].x, x[1][0].y, x[1][0].z, x[1][0].w};
            const uint32_t e0[4] = {s0.x, s0.y, s0.z, s0.w}, e1[4] = {s1.x, s1.y, s1.z, s1.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {         // slots k and k + 8
                const int sh = 16 * (k & 1);
                const float2 x0 = h2_to_f2(e4m3x2_to_h2(c0[k >> 1] >> sh)), x1 = h2_to_f2(e4m3x2_to_h2(c1[k >> 1] >> sh));
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float y0 = (u ? x0.y : x0.x) * exp_byte((e0[k >> 1] >> (sh + 8 * u)) & 255u);
                    const float y1 = (u ? x1.y : x1.x) * exp_byte((e1[k >> 1] >> (sh + 8 * u)) & 255u);
                    // exact in bf16: four significant bits
                    w[k + 8 * u] = (__float_as_uint(y0) >> 16) | (__float_as_uint(y1) & 0xffff0000u);
                }
            }
        } else {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const uint4 u = x[0][hf * (N - 1)], v = x[1][hf * (N - 1)];
                const uint32_t c0[4] = {u.x, u.y, u.z, u.w}, c1[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 8; ++k) w[8 * hf + k] = __byte_perm(c0[k >> 1], c1[k >> 1], k & 1 ? 0x7632 : 0x5410);
            }
        }
        const bool one = e + 1 >= p.E;
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            if (t < g.t0 || t >= g.t1) continue;
            __nv_bfloat16 *r = p.rec + (long long)t * p.E + e;
            if (VEC) {
                *reinterpret_cast<uint32_t *>(r) = w[t];
            } else {
                r[0] = __ushort_as_bfloat16((unsigned short)(w[t] & 0xffffu));
                if (!one) r[1] = __ushort_as_bfloat16((unsigned short)(w[t] >> 16));
            }
        }
    };
    const Plane k = plane(true), v = plane(false);
    for (int e = 2 * tid; e < max(k.E, v.E); e += 2 * threads) {
        uint4 xk[2][N], xv[2][N], sk, sv;
        load(k, e, xk, sk);
        load(v, e, xv, sv);
        emit(k, e, xk, sk);
        emit(v, e, xv, sv);
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

// Threads: one per pair of a record's elements (512 at most: longer records take several
// pieces), so that short records leave few threads idle.
int threads_of(const WriteArgs &a) {
    const int pairs = (a.ek > a.ev ? a.ek : a.ev) / 2 + 1;
    return std::min(kMaxThreads, (pairs + 31) / 32 * 32);
}

// Calls launch(e4m3, vec) as compile-time constants.
template <class Launch>
void by_format(bool e4m3, bool vec, Launch launch) {
    if (e4m3)
        vec ? launch(std::true_type{}, std::true_type{}) : launch(std::true_type{}, std::false_type{});
    else
        vec ? launch(std::false_type{}, std::true_type{}) : launch(std::false_type{}, std::false_type{});
}

// n rows of one sequence touch at most (n + 14) / 16 + 1 groups
unsigned write_groups(int batch, int n_rows) { return (unsigned)(((long long)n_rows + 14ll * batch) / 16 + batch); }

}  // namespace

cudaError_t launch_paged_append(const PagedShape &s, int batch, int n_rows, const void *kf, const void *vf,
                                const int32_t *cu, const int32_t *start, void *kpool, void *vpool,
                                const RopeTable &rope, int *err, cudaStream_t st) {
    WriteArgs a = write_args(s, batch, n_rows, cu, start, err);
    a.kf = const_cast<__nv_bfloat16 *>(static_cast<const __nv_bfloat16 *>(kf));
    a.vf = const_cast<__nv_bfloat16 *>(static_cast<const __nv_bfloat16 *>(vf));
    a.kpool = static_cast<unsigned char *>(kpool);
    a.vpool = static_cast<unsigned char *>(vpool);
    const dim3 grid(write_groups(batch, n_rows), 2);                    // (y: the plane)
    const bool vec = a.ek % 2 == 0 && a.ev % 2 == 0 && a.ak % 2 == 0 && a.av % 2 == 0;
    const size_t smem = (size_t)(a.d2 / 2) * 16 * sizeof(float2);       // at most 16 KB
    by_format(s.pool.e4m3 != 0, vec, [&](auto e4m3, auto v) {
        paged_append_kernel<decltype(e4m3)::value, decltype(v)::value><<<grid, threads_of(a), smem, st>>>(a, rope);
    });
    return cudaGetLastError();
}

cudaError_t launch_paged_read(const PagedShape &s, int batch, int n_rows, const int32_t *cu, const int32_t *start,
                              void *kf, void *vf, int *err, cudaStream_t st) {
    WriteArgs a = write_args(s, batch, n_rows, cu, start, err);
    a.kf = static_cast<__nv_bfloat16 *>(kf);
    a.vf = static_cast<__nv_bfloat16 *>(vf);
    const unsigned grid = write_groups(batch, n_rows);
    by_format(s.pool.e4m3 != 0, a.ek % 2 == 0 && a.ev % 2 == 0, [&](auto e4m3, auto v) {
        paged_read_kernel<decltype(e4m3)::value, decltype(v)::value><<<grid, threads_of(a), 0, st>>>(a);
    });
    return cudaGetLastError();
}

}  // namespace kpa
