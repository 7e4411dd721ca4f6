// fv_rmsnorm.cu -- root-mean-square norm with the residual's addition, 8-bit output with scales, and
// its gradient (sm_100a).  Definitions, layouts and errors: fastvim_ssm.h.
//
// Per row of E channels:  s = x + r,  y = w s rstd,  rstd = 1 / sqrt(mean(s^2) + eps).
// A row is read once: a group of G threads (32 .. 1024, one row per group) holds it in registers as
// NV vectors of V values a thread, so the kernel's traffic is its floor (x and r in, s and y out) and
// the copy rate bounds it.  Everything between load and store is fp32.  65536 rows of 1536 bf16 channels
// with an fp32 stream, 8-bit output with a scale for 128, into buffers that the caller keeps: 172 us, 0.99 of a 6.53
// TB/s copy; 65536 x 768 with bf16 output 92 us (1.0), without a residual 35 us (0.89: a row's fewer bytes are in
// flight), to 8 bits 38 us (0.61).
#include <cuda_fp8.h>

#include "fv_common.cuh"
#include "fv_host.cuh"
#include "fv_types.cuh"

namespace fv {
namespace {

struct RmsParams {
    long long M, x_stride;
    int E, block;  // block: channels per scale (0: one scale a row)
    float eps;
    const void *x, *r;
    const float* w;
    void *y, *s;
    float* scales;
};

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126: an all-zero block still has a finite inverse scale

// Sum over a group of G consecutive threads, known to all of them; groups are whole warps, and every
// thread of the block takes part.  `red`: blockDim.x / 32 floats, reusable after the next barrier pair.
template <int G>
__device__ __forceinline__ float group_sum(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (G > 32) {
        constexpr int kW = G / 32;
        const int warp = threadIdx.x >> 5;
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[warp] = v;
        __syncthreads();
        const int first = warp / kW * kW;
        v = 0.f;
#pragma unroll
        for (int i = 0; i < kW; ++i) v += red[first + i];
    }
    return v;
}
// Two sums at once.
template <int G>
__device__ __forceinline__ float2 group_sum(float2 v, float2* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if constexpr (G > 32) {
        constexpr int kW = G / 32;
        const int warp = threadIdx.x >> 5;
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[warp] = v;
        __syncthreads();
        const int first = warp / kW * kW;
        v = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            const float2 u = red[first + i];
            v.x += u.x;
            v.y += u.y;
        }
    }
    return v;
}
// Magnitudes are compared as whole numbers, which order them alike and put a NaN above all.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v, float* red) {
    v = __reduce_max_sync(0xffffffffu, v);
    if constexpr (G > 32) {
        constexpr int kW = G / 32;
        const int warp = threadIdx.x >> 5;
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[warp] = __uint_as_float(v);
        __syncthreads();
        const int first = warp / kW * kW;
        v = 0;
#pragma unroll
        for (int i = 0; i < kW; ++i) v = max(v, __float_as_uint(red[first + i]));
    }
    return v;
}
// The scale of values up to `most` (a magnitude): the smallest normal number stands for an all-zero block, a
// NaN stays one.
__device__ __forceinline__ float scale_of(uint32_t most) {
    const float s = __uint_as_float(most) / kE4m3Max;
    return s < kMinScale ? kMinScale : s;
}

// OUT: 0 = y in TX, 1 = e4m3 with scales.  TX: x (and y), TR: the residual stream (RES) -- r and s.
template <typename TX, typename TR, bool RES, int OUT, int V, int G, int NV>
__global__ void __launch_bounds__(G < 128 ? 128 : G) rms_norm_kernel(RmsParams p) {
    constexpr int kBlock = G < 128 ? 128 : G;
    __shared__ float red[kBlock / 32];
    const int t = threadIdx.x % G;
    const long long row = (long long)blockIdx.x * (kBlock / G) + threadIdx.x / G;
    const bool live = row < p.M;
    const int nvec = p.E / V;
    const TX* x = (const TX*)p.x + (live ? row * p.x_stride : 0);
    const size_t at = live ? (size_t)row * p.E : 0;
    float s[NV][V];
    float r[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + G * i) * V;
#pragma unroll
        for (int j = 0; j < V; ++j) s[i][j] = r[i][j] = 0.f;
        if (live && t + G * i < nvec) {
            load_vec<TX, V, true>(x + c, s[i]);
            if constexpr (RES) load_vec<TR, V, true>((const TR*)p.r + at + c, r[i]);
        }
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s[i][j] += r[i][j];
            q = fmaf(s[i][j], s[i][j], q);
        }
    if constexpr (RES) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && t + G * i < nvec) store_vec<TR, V>((TR*)p.s + at + (t + G * i) * V, s[i]);
    }
    const float rstd = rsqrtf(group_sum<G>(q, red) / (float)p.E + p.eps);
    uint32_t most = 0;  // one scale a row
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + G * i) * V;
        const bool in = live && t + G * i < nvec;
        if (in) {
            float w[V];
            load_vec<float, V, false>(p.w + c, w);
#pragma unroll
            for (int j = 0; j < V; ++j) s[i][j] = s[i][j] * rstd * w[j];
            if constexpr (OUT == 0) store_vec<TX, V>((TX*)p.y + at + c, s[i]);
        }
        if constexpr (OUT == 1) {
            if (p.block == 0)
#pragma unroll
                for (int j = 0; j < V; ++j) most = max(most, magnitude(s[i][j]));
        }
    }
    if constexpr (OUT == 1) {
        uint8_t* y = (uint8_t*)p.y + at;
        auto quantise = [&](int i, float inv) {
            uint32_t o[V / 4];
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(s[i][j] * inv, s[i][j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(s[i][j + 2] * inv, s[i][j + 3] * inv), __NV_SATFINITE, __NV_E4M3);
                o[j / 4] = lo | hi << 16;
            }
            if (live && t + G * i < nvec) {
                if constexpr (V == 8)
                    __stcs(reinterpret_cast<uint2*>(y + (t + G * i) * V), make_uint2(o[0], o[1]));
                else
                    __stcs(reinterpret_cast<uint32_t*>(y + (t + G * i) * V), o[0]);
            }
        };
        if (p.block == 0) {
            const float scale = scale_of(group_max<G>(most, red));
            if (live && t == 0) p.scales[row] = scale;
            const float inv = 1.f / scale;
#pragma unroll
            for (int i = 0; i < NV; ++i) quantise(i, inv);
        } else {
            // 128 channels are the vectors of 128 / V neighbouring lanes (E is a multiple of 128 here)
            constexpr int kL = 128 / V;
            const int nb = p.E / 128;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < V; ++j) m = max(m, magnitude(s[i][j]));
#pragma unroll
                for (int o = kL / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                const float scale = scale_of(m);
                if (live && t + G * i < nvec && (t & (kL - 1)) == 0) p.scales[(size_t)row * nb + (t + G * i) / kL] = scale;
                quantise(i, 1.f / scale);
            }
        }
    }
}

// ---- gradient --------------------------------------------------------------------------------------
// With n = s rstd and c = w dy:  ds = rstd (c - n mean(n c)) + ds_up,  dw = sum over rows of n dy.
// Blocks walk the rows (row groups blockIdx.x, + gridDim.x, ..); each thread keeps its channels' share
// of dw in registers, the block's groups add theirs in order, and a second kernel adds the blocks' in
// order, so the sums do not depend on timing.  65536 x 768, bf16 with an fp32 stream: 136 us with ds (805 MB, 0.9 of
// the copy rate), 110 us without (604 MB, 0.84); all bf16 76 and 65 us (403 and 302 MB, 0.81 and 0.71): bound by
// the latency between a row's loads and its sums.
struct RmsGradParams {
    long long M;
    int E;
    float eps;
    const void *s, *dy, *ds;
    const float* w;
    void *dx, *dr;  // dx in the type of dy; dr (may be null) in the type of s
    float* part;    // [gridDim.x][E]
};

// Blocks on an SM at once, by the registers that a thread's part of a row takes.
template <int G, int VALUES>
constexpr int grad_on_sm() { return G > 256 || VALUES > 24 ? 1 : VALUES > 8 ? 2 : 4; }

template <typename TY, typename TS, int V, int G, int NV>
__global__ void __launch_bounds__(G < 256 ? 256 : G, grad_on_sm<G, V * NV>()) rms_grad_kernel(RmsGradParams p) {
    constexpr int kBlock = G < 256 ? 256 : G, kRows = kBlock / G;
    // The next rows' loads are in flight while this row's sums are made, where the registers hold them (bf16
    // throughout, 16384 x 4096: 82 us, without 103 us; fp32 throughout, one vector, 65536 x 1024: 138 us without, 162 us
    // with them).
    constexpr int kHeld = NV * V * (int)(sizeof(TS) + sizeof(TY));
    constexpr bool kAhead = NV * V <= 8 ? kHeld <= 32 : NV * V <= 16 && kHeld <= 96;
    __shared__ float2 red[kBlock / 32];
    extern __shared__ float dw_sm[];  // [kRows][E] with kRows > 1
    const int t = threadIdx.x % G, grp = threadIdx.x / G;
    const int nvec = p.E / V;
    const float inv_e = 1.f / (float)p.E;
    float dw[NV][V];
    Raw<TS, V> rs[NV];
    Raw<TY, V> rc[NV];
    auto fetch = [&](long long row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = row < p.M && t + G * i < nvec;
            const size_t at = (size_t)row * p.E + (t + G * i) * V;
            rs[i].load((const TS*)p.s + at, in);
            rc[i].load((const TY*)p.dy + at, in);
        }
    };
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) dw[i][j] = 0.f;
    const long long step = (long long)gridDim.x * kRows;
    if (kAhead) fetch((long long)blockIdx.x * kRows + grp);
    for (long long first = (long long)blockIdx.x * kRows; first < p.M; first += step) {
        const long long row = first + grp;
        const bool live = row < p.M;
        const size_t at = live ? (size_t)row * p.E : 0;
        if (!kAhead) fetch(row);
        float s[NV][V], c[NV][V], up[NV][V];
        float2 sums = make_float2(0.f, 0.f);  // of s s and of s w dy
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            rs[i].unpack(s[i]);
            rc[i].unpack(c[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) up[i][j] = 0.f;
            if (p.ds && live && t + G * i < nvec) load_vec<TS, V, true>((const TS*)p.ds + at + (t + G * i) * V, up[i]);
        }
        if (kAhead) fetch(row + step);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float w[V];
#pragma unroll
            for (int j = 0; j < V; ++j) w[j] = 0.f;
            if (t + G * i < nvec) load_vec<float, V, false>(p.w + (t + G * i) * V, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                sums.x = fmaf(s[i][j], s[i][j], sums.x);
                sums.y = fmaf(s[i][j], c[i][j] * w[j], sums.y);
            }
        }
        sums = group_sum<G>(sums, red);
        const float rstd = rsqrtf(sums.x * inv_e + p.eps);
        const float k = sums.y * inv_e * rstd * rstd;  // mean(n c) rstd
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (t + G * i) * V;
            if (live && t + G * i < nvec) {
                float w[V];
                load_vec<float, V, false>(p.w + col, w);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    dw[i][j] = fmaf(s[i][j] * rstd, c[i][j], dw[i][j]);
                    up[i][j] += rstd * (c[i][j] * w[j] - s[i][j] * k);
                }
                store_vec<TY, V>((TY*)p.dx + at + col, up[i]);
                if (p.dr) store_vec<TS, V>((TS*)p.dr + at + col, up[i]);
            }
        }
    }
    float* part = p.part + (size_t)blockIdx.x * p.E;
    if constexpr (kRows == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (t + G * i < nvec)
#pragma unroll
                for (int j = 0; j < V; ++j) part[(t + G * i) * V + j] = dw[i][j];
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (t + G * i < nvec)
#pragma unroll
                for (int j = 0; j < V; ++j) dw_sm[(size_t)grp * p.E + (t + G * i) * V + j] = dw[i][j];
        __syncthreads();
        for (int c = threadIdx.x; c < p.E; c += kBlock) {
            float a = 0.f;
#pragma unroll
            for (int g = 0; g < kRows; ++g) a += dw_sm[(size_t)g * p.E + c];
            part[c] = a;
        }
    }
}

// out[c] = sum over n partial rows, added in a fixed order: thread (c, g) takes rows g, g + 32, ..,
// and the 32 sums of a column are added in order.  Block: 32 columns x 32 row groups.
__global__ void __launch_bounds__(1024) rms_grad_reduce_kernel(const float* __restrict__ part, int n, int E,
                                                                float* __restrict__ out) {
    __shared__ float sm[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float a = 0.f;
    if (c < E)
#pragma unroll 4
        for (int i = threadIdx.y; i < n; i += 32) a += part[(size_t)i * E + c];
    sm[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y == 0 && c < E) {
        a = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) a += sm[i][threadIdx.x];
        out[c] = a;
    }
}

// ---- host ------------------------------------------------------------------------------------------
constexpr int kMaxE = 16384;
size_t type_size(int t) { return t == FV_TYPE_F32 ? 4 : t == FV_TYPE_E4M3 ? 1 : 2; }
bool io_type(int t) { return t == FV_TYPE_F32 || t == FV_TYPE_BF16 || t == FV_TYPE_F16; }

fv_status check_rms(const fv_rmsnorm_args* a) {
    if (!a) return FV_ERR_NULL;
    if (a->M < 0 || a->E < 4 || a->E % 4 != 0) return FV_ERR_SHAPE;
    if (!io_type(a->x_type)) return FV_ERR_SHAPE;
    if (a->y_type != a->x_type && a->y_type != FV_TYPE_E4M3) return FV_ERR_SHAPE;
    if (a->residual && a->res_type != FV_TYPE_F32 && a->res_type != a->x_type) return FV_ERR_SHAPE;
    if (a->block != 0 && (a->block != 128 || a->E % 128 != 0 || a->y_type != FV_TYPE_E4M3)) return FV_ERR_SHAPE;
    if (a->x_stride != 0 && (a->x_stride < a->E || a->x_stride % 4 != 0)) return FV_ERR_SHAPE;
    if (!(a->eps > 0.f && a->eps <= 3.0e38f)) return FV_ERR_SHAPE;
    if (a->E > kMaxE || a->M >= (1ll << 31)) return FV_ERR_UNSUPPORTED;
    if (!a->weight) return FV_ERR_NULL;
    if (a->M > 0 && (!a->x || !a->y)) return FV_ERR_NULL;
    if (a->M > 0 && a->residual && !a->s) return FV_ERR_NULL;
    if (!a->residual && a->s) return FV_ERR_SHAPE;
    if (a->M > 0 && a->y_type == FV_TYPE_E4M3 && !a->scales) return FV_ERR_NULL;
    if (a->y_type != FV_TYPE_E4M3 && a->scales) return FV_ERR_SHAPE;
    const void* ps[] = {a->x, a->residual, a->weight, a->y, a->s, a->scales};
    for (const void* p : ps)
        if (!ptr_aligned16(p)) return FV_ERR_ALIGN;
    const size_t xb = type_size(a->x_type), xs = a->x_stride ? (size_t)a->x_stride : (size_t)a->E;
    if (a->M > 0) {
        const size_t n = (size_t)a->M * a->E, nx = ((size_t)(a->M - 1) * xs + a->E) * xb;
        const size_t ny = n * type_size(a->y_type), nr = n * type_size(a->res_type);
        const size_t nsc = (size_t)a->M * (a->block ? a->E / a->block : 1) * 4;
        const void* out[] = {a->y, a->s, a->scales};
        const size_t no[] = {ny, a->residual ? nr : 0, nsc};
        for (int i = 0; i < 3; ++i) {
            if (ranges_overlap(out[i], no[i], a->weight, (size_t)a->E * 4)) return FV_ERR_ALIAS;
            for (int j = i + 1; j < 3; ++j)
                if (ranges_overlap(out[i], no[i], out[j], no[j])) return FV_ERR_ALIAS;
            // s may be the residual itself (each value is read before it is written); nothing else overlaps
            if (ranges_overlap(out[i], no[i], a->x, nx)) return FV_ERR_ALIAS;
            if (ranges_overlap(out[i], no[i], a->residual, nr) && !(i == 1 && a->s == a->residual)) return FV_ERR_ALIAS;
        }
    }
    return FV_OK;
}

// 8-value vectors where rows start on 8 values, else 4-value ones.
int vec_of(int E, long long stride) { return (E % 8 == 0 && stride % 8 == 0) ? 8 : 4; }

template <typename TX, typename TR, bool RES, int OUT, int V, int G, int NV>
fv_status launch_rms(const RmsParams& p, cudaStream_t st) {
    constexpr int kBlock = G < 128 ? 128 : G;
    const long long rows = kBlock / G;
    rms_norm_kernel<TX, TR, RES, OUT, V, G, NV><<<(unsigned)((p.M + rows - 1) / rows), kBlock, 0, st>>>(p);
    return launch_status("rms_norm_kernel");
}

// The group of threads that holds a row.  One warp a row needs no barrier, and a short row in few registers
// keeps many rows in flight on an SM; with a residual twice the loads are in flight, so fewer vectors a
// thread do: 65536 rows of 768 channels take 93 us in warps of 3 vectors, 91 us in 128 threads of one (8-bit
// output 93 and 85 us), without a residual 34 and 45 us; half as wide vectors gain nothing (131072 x 380: 95
// and 104 us).  8192 rows of 8192: 123 us in 512 threads of 2 vectors, 134 us in 256 of 4, without a residual 56 and
// 44 us.  4096 rows of 16384: 139 us in 1024 of 2, 160 us in 512 of 4, without a residual 61 and 52 us.
template <typename TX, typename TR, bool RES, int OUT, int V>
fv_status rms_by_width(const RmsParams& p, cudaStream_t st) {
    const int n = p.E / V;
    if (n <= 32) return launch_rms<TX, TR, RES, OUT, V, 32, 1>(p, st);
    if (n <= 64) return launch_rms<TX, TR, RES, OUT, V, 32, 2>(p, st);
    if constexpr (RES && V == 8) {
        if (n <= 128) return launch_rms<TX, TR, RES, OUT, V, 128, 1>(p, st);
    } else {
        if (n <= 96) return launch_rms<TX, TR, RES, OUT, V, 32, 3>(p, st);
        if (n <= 128) return launch_rms<TX, TR, RES, OUT, V, 64, 2>(p, st);
    }
    if (n <= 192) return launch_rms<TX, TR, RES, OUT, V, 64, 3>(p, st);
    if (n <= 256) return launch_rms<TX, TR, RES, OUT, V, 128, 2>(p, st);
    if (n <= 512) return launch_rms<TX, TR, RES, OUT, V, 256, 2>(p, st);
    if constexpr (RES) {
        if (n <= 1024) return launch_rms<TX, TR, RES, OUT, V, 512, 2>(p, st);
        if (n <= 2048) return launch_rms<TX, TR, RES, OUT, V, 1024, 2>(p, st);
    } else {
        if (n <= 1024) return launch_rms<TX, TR, RES, OUT, V, 256, 4>(p, st);
        if (n <= 2048) return launch_rms<TX, TR, RES, OUT, V, 512, 4>(p, st);
    }
    if constexpr (V == 4) return launch_rms<TX, TR, RES, OUT, V, 1024, 4>(p, st);
    return FV_ERR_UNSUPPORTED;  // E <= 16384
}
template <typename TX, typename TR, bool RES>
fv_status rms_by_out(const RmsParams& p, bool fp8, int V, cudaStream_t st) {
    if (fp8) return V == 8 ? rms_by_width<TX, TR, RES, 1, 8>(p, st) : rms_by_width<TX, TR, RES, 1, 4>(p, st);
    return V == 8 ? rms_by_width<TX, TR, RES, 0, 8>(p, st) : rms_by_width<TX, TR, RES, 0, 4>(p, st);
}
template <typename TX>
fv_status rms_by_res(const RmsParams& p, bool res, bool res_f32, bool fp8, int V, cudaStream_t st) {
    if (!res) return rms_by_out<TX, TX, false>(p, fp8, V, st);
    if (res_f32) return rms_by_out<TX, float, true>(p, fp8, V, st);
    return rms_by_out<TX, TX, true>(p, fp8, V, st);
}

fv_status check_rms_grad(const fv_rmsnorm_grad_args* a) {
    if (!a) return FV_ERR_NULL;
    if (a->M < 0 || a->E < 4 || a->E % 4 != 0) return FV_ERR_SHAPE;
    if (!io_type(a->y_type)) return FV_ERR_SHAPE;
    if (a->s_type != FV_TYPE_F32 && a->s_type != a->y_type) return FV_ERR_SHAPE;
    if (!(a->eps > 0.f && a->eps <= 3.0e38f)) return FV_ERR_SHAPE;
    if (a->E > kMaxE || a->M >= (1ll << 31)) return FV_ERR_UNSUPPORTED;
    if (!a->weight || !a->dweight) return FV_ERR_NULL;
    if (a->M > 0 && (!a->s || !a->dy || !a->dx)) return FV_ERR_NULL;
    const void* ps[] = {a->s, a->dy, a->ds, a->weight, a->dx, a->dresidual, a->dweight};
    for (const void* p : ps)
        if (!ptr_aligned16(p)) return FV_ERR_ALIGN;
    const size_t n = (size_t)a->M * a->E, ny = n * type_size(a->y_type), ns = n * type_size(a->s_type), nw = (size_t)a->E * 4;
    const void* out[] = {a->dx, a->dresidual, a->dweight};
    const size_t no[] = {ny, ns, nw};
    const void* in[] = {a->s, a->dy, a->ds, a->weight};
    const size_t ni[] = {ns, ny, ns, nw};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 4; ++j)
            if (ranges_overlap(out[i], no[i], in[j], ni[j])) return FV_ERR_ALIAS;
        for (int j = i + 1; j < 3; ++j)
            if (ranges_overlap(out[i], no[i], out[j], no[j])) return FV_ERR_ALIAS;
    }
    return FV_OK;
}

// Blocks of the gradient: those that the registers let stand on an SM at once (148 SMs), so that none starts
// when others end, and no more than there are row groups.  bf16 with an fp32 stream and ds, 65536 x 1536 (two on an SM):
// 261 us with 296 blocks, 265 us with 592, 317 us with 148; 131072 x 200 (four): 78 us with 592, 77 and 92 us with
// twice and half as many; 65536 x 768 136, 131 and 155 us.
constexpr int kMostBlocks = 148 * 4;
int grad_blocks(long long M, int rows, int most) {
    const long long groups = (M + rows - 1) / rows;
    return (int)(groups < most ? (groups < 1 ? 1 : groups) : most);
}

template <typename TY, typename TS, int V, int G, int NV>
fv_status launch_grad(RmsGradParams p, float* dweight, cudaStream_t st) {
    constexpr int kBlock = G < 256 ? 256 : G, kRows = kBlock / G;
    const int nb = grad_blocks(p.M, kRows, 148 * grad_on_sm<G, V * NV>());
    static_assert(kRows == 1 || kRows * G * NV * V * 4 <= 48 * 1024, "dw_sm needs no opt-in");
    const size_t smem = kRows > 1 ? (size_t)kRows * p.E * 4 : 0;
    rms_grad_kernel<TY, TS, V, G, NV><<<nb, kBlock, smem, st>>>(p);
    const fv_status s = launch_status("rms_grad_kernel");
    if (s != FV_OK) return s;
    rms_grad_reduce_kernel<<<(p.E + 31) / 32, dim3(32, 32), 0, st>>>(p.part, nb, p.E, dweight);
    return launch_status("rms_grad_reduce_kernel");
}
// How many threads hold a row (without and with ds): more of them keep more loads in flight, fewer wait less for one
// another.  16-bit dy take two vectors a thread, all fp32 one: bf16 with a bf16 stream, 65536 x 1024: 81 and 95 us in 64
// threads of 2, 90 and 97 us in 128 of one; 32768 x 2048: 81 and 97, 89 and 117; with an fp32 stream 137 and 179, 146
// and 176; 142 and 174, 146 and 172; all fp32 147 and 177, 138 and 170; 146 and 176, 139 and 168.  Rows of 12288 bytes
// and more, in 512 threads of 2 vectors or 256 of 4: bf16, 16384 x 8192: 157 and 180, 239 and 259; with an fp32
// stream 257 and 341, 362 and 378; all fp32, of 4096 channels on, 347 and 372, 319 and 357; 4-value vectors 32768 x
// 2052: 172 and 188, 113 and 138.  4096 x 16384, fp32 stream: 192 and 203 us in 512 of 4, 286 and 318 in 1024 of 2.
template <typename TY, typename TS, int V>
fv_status grad_by_width(const RmsGradParams& p, float* dw, cudaStream_t st) {
    const int n = p.E / V;
    if (n <= 32) return launch_grad<TY, TS, V, 32, 1>(p, dw, st);
    if (n <= 64) return launch_grad<TY, TS, V, 32, 2>(p, dw, st);
    if (n <= 96) return launch_grad<TY, TS, V, 32, 3>(p, dw, st);
    if constexpr (sizeof(TY) == 4) {
        if (n <= 128) return launch_grad<TY, TS, V, 128, 1>(p, dw, st);
        if (n <= 192) return launch_grad<TY, TS, V, 64, 3>(p, dw, st);
        if (n <= 256) return launch_grad<TY, TS, V, 256, 1>(p, dw, st);
    } else {
        if (n <= 128) return launch_grad<TY, TS, V, 64, 2>(p, dw, st);
        if (n <= 192) return launch_grad<TY, TS, V, 64, 3>(p, dw, st);
        if (n <= 256) return launch_grad<TY, TS, V, 128, 2>(p, dw, st);
    }
    if (n <= 512) return launch_grad<TY, TS, V, 256, 2>(p, dw, st);
    if constexpr (sizeof(TY) == 2 && V == 8) {
        if (n <= 1024) return launch_grad<TY, TS, V, 512, 2>(p, dw, st);
    } else {
        if (n <= 1024) return launch_grad<TY, TS, V, 256, 4>(p, dw, st);
    }
    if (n <= 2048) return launch_grad<TY, TS, V, 512, 4>(p, dw, st);
    if constexpr (V == 4) return launch_grad<TY, TS, V, 1024, 4>(p, dw, st);
    return FV_ERR_UNSUPPORTED;  // E <= 16384
}
template <typename TY, typename TS>
fv_status grad_by_vec(const RmsGradParams& p, float* dw, cudaStream_t st) {
    return vec_of(p.E, p.E) == 8 ? grad_by_width<TY, TS, 8>(p, dw, st) : grad_by_width<TY, TS, 4>(p, dw, st);
}

}  // namespace
}  // namespace fv

extern "C" {

fv_status fastvim_rmsnorm_validate(const fv_rmsnorm_args* args) { return fv::check_rms(args); }

fv_status fastvim_rmsnorm_forward(const fv_rmsnorm_args* args, void* stream) {
    fv_status s = fv::check_rms(args);
    if (s != FV_OK || args->M == 0) return s;
    const fv_rmsnorm_args& a = *args;
    const long long xs = a.x_stride ? a.x_stride : a.E;
    const fv::RmsParams p{a.M, xs, a.E, a.block, a.eps, a.x, a.residual, a.weight, a.y, a.s, a.scales};
    const int V = fv::vec_of(a.E, xs);
    const bool res = a.residual != nullptr, f32 = a.res_type == FV_TYPE_F32, fp8 = a.y_type == FV_TYPE_E4M3;
    cudaStream_t st = (cudaStream_t)stream;
    if (a.x_type == FV_TYPE_F32) {
        return res ? fv::rms_by_out<float, float, true>(p, fp8, V, st) : fv::rms_by_out<float, float, false>(p, fp8, V, st);
    }
    if (a.x_type == FV_TYPE_BF16) return fv::rms_by_res<__nv_bfloat16>(p, res, f32, fp8, V, st);
    return fv::rms_by_res<__half>(p, res, f32, fp8, V, st);
}

size_t fastvim_rmsnorm_backward_workspace_size(const fv_rmsnorm_grad_args* args) {
    if (!args || args->M < 0 || args->E < 4 || args->E % 4 != 0 || args->E > fv::kMaxE) return 0;
    return fv::round_up256((size_t)fv::grad_blocks(args->M, 1, fv::kMostBlocks) * args->E * sizeof(float));
}

fv_status fastvim_rmsnorm_backward(const fv_rmsnorm_grad_args* args, void* ws, size_t ws_bytes, void* stream) {
    fv_status s = fv::check_rms_grad(args);
    if (s != FV_OK) return s;
    if (!ws || ((uintptr_t)ws & 255u) != 0 || ws_bytes < fastvim_rmsnorm_backward_workspace_size(args)) return FV_ERR_WORKSPACE;
    const fv_rmsnorm_grad_args& a = *args;
    const fv::RmsGradParams p{a.M, a.E, a.eps, a.s, a.dy, a.ds, a.weight, a.dx, a.dresidual, (float*)ws};
    cudaStream_t st = (cudaStream_t)stream;
    if (a.y_type == FV_TYPE_F32) return fv::grad_by_vec<float, float>(p, a.dweight, st);
    const bool f32 = a.s_type == FV_TYPE_F32;
    if (a.y_type == FV_TYPE_BF16)
        return f32 ? fv::grad_by_vec<__nv_bfloat16, float>(p, a.dweight, st)
                   : fv::grad_by_vec<__nv_bfloat16, __nv_bfloat16>(p, a.dweight, st);
    return f32 ? fv::grad_by_vec<__half, float>(p, a.dweight, st) : fv::grad_by_vec<__half, __half>(p, a.dweight, st);
}

}  // extern "C"
