// fv_linattn_simt.cuh -- linear attention on fp32 FMAs: the fp32 forward and gradient.
//
// Chunks of 64 tokens; every product of a chunk is a 64 x 64 (or 64 x dk) tile by 256 threads.  Warp w
// takes 32 rows x a quarter of the columns; lane l rows 8 i + l / 4 and neighbouring columns, so a tile's
// rows reach a warp as 8 + 4 conflict-free 16-byte loads for 64 FMAs a thread, issued as packed pairs.
// Bound by the FMA and shared-memory pipes (1 M FMAs a chunk and head of 64 x 64): 8 x 1024 tokens x 6 heads of
// 64 x 64 take 67 us forward, where the FMAs of its 768 chunks alone would take 22 us, and 148 us for the
// gradient; the shared-memory pipe is at 0.55 and 0.7 of its rate.
#pragma once

#include "fv_linattn.cuh"
#include "fv_tc.cuh"

namespace fv {
namespace la {

constexpr int kC = 64;        // tokens per chunk
constexpr int kThr = 256;
__host__ __device__ constexpr int row_stride(int d) { return d + 4; }
constexpr int kVS = row_stride(kTile);  // stride of 64-column tiles

// This thread's place in a 64-row tile of 4 * 4 * NJ columns.
struct Place {
    int r0, c4;  // rows r0 + 8 i; columns (4 wc + c4) * NJ + j
    int wr, wc;  // 32-row and column block of the warp
};
__device__ __forceinline__ Place place() {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Place p;
    p.wr = warp >> 2;
    p.wc = warp & 3;
    p.r0 = 32 * p.wr + (lane >> 2);
    p.c4 = 4 * p.wc + (lane & 3);
    return p;
}

// Column j of this thread in a token x token tile.
__device__ __forceinline__ int spread(const Place& p, int j) { return 16 * p.wc + (threadIdx.x & 3) + 4 * j; }

// Rows [0, kC) of columns [0, W) of a token-major tensor into sm (asynchronously); zeros behind the n rows and
// `cols` columns (a multiple of 8).
template <int W>
__device__ __forceinline__ void load_rows(float* sm, int stride, const float* src, long long token_stride, int n, int cols) {
#pragma unroll
    for (int i = threadIdx.x; i < kC * (W / 4); i += kThr) {
        const int r = i / (W / 4), c = (i % (W / 4)) * 4;
        const bool in = r < n && c < cols;
        cp_async16(sm + r * stride + c, in ? src + (long long)r * token_stride + c : src, in ? 16u : 0u);
    }
}
// ROWS x kTile columns of a [dk][dv] matrix, zeros without one
template <int ROWS>
__device__ __forceinline__ void load_state(float* sm, const float* src, int dk, int dv, int cols) {
#pragma unroll
    for (int i = threadIdx.x; i < ROWS * (kTile / 4); i += kThr) {
        const int r = i / (kTile / 4), c = (i % (kTile / 4)) * 4;
        const bool in = r < dk && c < cols;
        if (src) cp_async16(sm + r * kVS + c, in ? src + (size_t)r * dv + c : src, in ? 16u : 0u);
        else *reinterpret_cast<float4*>(sm + r * kVS + c) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

// acc[4][NJ] += A rows . B rows over K columns (both row-major): B's rows are the output's columns, NJ
// neighbouring ones a thread; SPREAD: 16 wc + lane % 4 + 4 j instead, whose loads meet no bank twice.
template <int NJ, bool SPREAD>
__device__ __forceinline__ void mm_nt(float (&acc)[4][NJ], const float* A, int as, const float* B, int bs, int K, const Place& p) {
    float2 s[4][NJ];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) s[i][j] = make_float2(0.f, 0.f);
    const float *a0 = A + p.r0 * as, *b0 = B + (SPREAD ? spread(p, 0) : p.c4 * NJ) * bs;
#pragma unroll 2
    for (int k = 0; k < K; k += 4) {
        float4 a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(a0 + 8 * i * as + k);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const float4 b = *reinterpret_cast<const float4*>(b0 + (SPREAD ? 4 * j : j) * bs + k);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[i][j] = tc::fma2(make_float2(a[i].x, a[i].y), make_float2(b.x, b.y), s[i][j]);
                s[i][j] = tc::fma2(make_float2(a[i].z, a[i].w), make_float2(b.z, b.w), s[i][j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] += s[i][j].x + s[i][j].y;
}
// acc[4][NJ] += A x B over k < K.
template <int NJ>
__device__ __forceinline__ void mm_nn(float (&acc)[4][NJ], const float* A, int as, const float* B, int bs, int K, const Place& p) {
    float2 s[4][NJ / 2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NJ / 2; ++j) s[i][j] = make_float2(acc[i][2 * j], acc[i][2 * j + 1]);
    const float *a0 = A + p.r0 * as, *b0 = B + p.c4 * NJ;
#pragma unroll 2
    for (int k = 0; k < K; k += 4) {
        float a[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(a0 + 8 * i * as + k);
            a[i][0] = v.x; a[i][1] = v.y; a[i][2] = v.z; a[i][3] = v.w;
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
            for (int j = 0; j < NJ; j += 4) {
                const float4 b = *reinterpret_cast<const float4*>(b0 + (k + t) * bs + j);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 aa = make_float2(a[i][t], a[i][t]);
                    s[i][j / 2] = tc::fma2(aa, make_float2(b.x, b.y), s[i][j / 2]);
                    s[i][j / 2 + 1] = tc::fma2(aa, make_float2(b.z, b.w), s[i][j / 2 + 1]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NJ / 2; ++j) {
            acc[i][2 * j] = s[i][j].x;
            acc[i][2 * j + 1] = s[i][j].y;
        }
}
// acc[R][4]: rows R ((lane / 4) + 8 (warp / 4)) + i, columns 4 c4 + j, += sum over tokens t of A[t][row] B[t][column].
template <int R>
__device__ __forceinline__ void mm_tn(float (&acc)[R][4], const float* A, int as, const float* B, int K, const Place& p) {
    float2 s[R][2];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        s[i][0] = make_float2(acc[i][0], acc[i][1]);
        s[i][1] = make_float2(acc[i][2], acc[i][3]);
    }
    const int row = R * (8 * p.wr + ((threadIdx.x & 31) >> 2));
#pragma unroll 4
    for (int t = 0; t < K; ++t) {
        const float4 b = *reinterpret_cast<const float4*>(B + t * kVS + 4 * p.c4);
#pragma unroll
        for (int i = 0; i < R; i += 4) {
            const float4 a = *reinterpret_cast<const float4*>(A + t * as + row + i);
            const float v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 aa = make_float2(v[e], v[e]);
                s[i + e][0] = tc::fma2(aa, make_float2(b.x, b.y), s[i + e][0]);
                s[i + e][1] = tc::fma2(aa, make_float2(b.z, b.w), s[i + e][1]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        acc[i][0] = s[i][0].x;
        acc[i][1] = s[i][0].y;
        acc[i][2] = s[i][1].x;
        acc[i][3] = s[i][1].y;
    }
}

// Exponents of a chunk, by one warp, two tokens a lane (fractions in units of 2^-24: 64 of them fit 32 bits);
// tokens behind the n-th keep the last sum.
__device__ __forceinline__ void chunk_exponents(const Shape& sh, const float* g, int h, int row, int n, Exponent* e) {
    const int lane = threadIdx.x & 31;
    FixedSum f[2];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        const float v = t < n ? __ldg(g + (sh.head_decay ? h : (long long)(row + t) * sh.gs + h)) : 0.f;
        bad |= v != v;
        f[i] = fixed_exponent<24>(v);
    }
    FixedSum s{f[0].hi + f[1].hi, f[0].lo + f[1].lo, f[0].rest + f[1].rest};
    warp_scan(s);
    bad = __any_sync(0xffffffffu, bad);
    e[2 * lane] = exponent_of<24>(s.hi - f[1].hi, s.lo - f[1].lo, bad ? __int_as_float(0x7fffffff) : s.rest - f[1].rest);
    e[2 * lane + 1] = exponent_of<24>(s.hi, s.lo, bad ? __int_as_float(0x7fffffff) : s.rest);
}
__device__ __forceinline__ float weight_of(const Exponent& e) { return ex2_approx(e.hi + e.lo); }

// ---- forward ----------------------------------------------------------------------------------------
// DK: dk rounded up to 64 or 128.  P takes Q's place and the weighted v takes v's.
template <int DK>
constexpr size_t fwd_smem() {
    return (size_t)(2 * kC * row_stride(DK) + kC * kVS + DK * kVS) * 4 + kC * sizeof(Exponent);
}

// One piece, head and 64 columns of v: walks the piece's chunks with the state in shared memory.
// OUT: writes y (and, behind a sequence of one piece, the final state).  Without it: the piece's own state
// from zero into st_loc and its decay into piece_decay.
template <int DK, bool OUT>
__global__ void __launch_bounds__(kThr, DK == 64 ? (OUT ? 2 : 3) : 1)
simt_kernel(Shape sh, PackedPlan plan, Tensors x, const float* start, float* st_loc, float* piece_decay, unsigned* status) {
    if (!sh.packed && blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
    extern __shared__ __align__(16) float sm[];
    constexpr int QS = row_stride(DK), R = DK / 16;
    float* Q = sm;
    float* K = Q + kC * QS;
    float* V = K + kC * QS;
    float* S = V + kC * kVS;
    Exponent* ex = reinterpret_cast<Exponent*>(S + DK * kVS);
    Piece pc;
    const int tiles = (sh.dv + kTile - 1) / kTile, per = sh.H * tiles, hy = blockIdx.x % per;
    int id;
    if (!get_piece(sh, plan, blockIdx.x / per, pc, id)) return wait_for_primary();  // no launch ends before those it overlaps
    // a piece's own state is needed where another follows, or where its sequence's final state is asked for;
    // a sequence of one piece carries its state alone
    if (!OUT && (pc.flags == 3 || ((pc.flags & 2) && (!x.st || sh.look_back)))) return;
    const bool last_state = x.st && (sh.look_back ? (pc.flags & 2) : pc.flags == 3);
    const int h = hy / tiles, c0 = (hy - h * tiles) * kTile;
    const int hk = key_head(sh, h), cols = min(kTile, sh.dv - c0);
    const Place p = place();
    const int c = 4 * p.c4;               // this thread's four columns
    const bool live = 16 * p.wc < cols;   // this warp's columns
    const int srow = R * (8 * p.wr + ((threadIdx.x & 31) >> 2));
    const size_t state_at = ((size_t)id * sh.H + h) * sh.dk * sh.dv;
    const float* s_in = !OUT ? nullptr : pc.flags != 3 ? start + state_at
                        : x.s0 ? x.s0 + ((size_t)pc.seq * sh.H + h) * sh.dk * sh.dv : nullptr;
    if (!OUT) launch_dependents();  // the outputs' blocks may begin with their loads and scores
    auto enter = [&]() {            // the state entering the piece
        if (OUT) wait_for_primary();
        if (OUT && sh.look_back && pc.flags != 3) {
            for (int i = threadIdx.x; i < DK * (kTile / 4); i += kThr) {
                const int r = i / (kTile / 4), k = (i % (kTile / 4)) * 4;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < sh.dk && k < cols) v = look_back(sh, start, piece_decay, x.s0, id, pc.seq, h, (size_t)r * sh.dv + c0 + k);
                *reinterpret_cast<float4*>(S + r * kVS + k) = v;
            }
        } else {
            load_state<DK>(S, s_in ? s_in + c0 : nullptr, sh.dk, sh.dv, cols);
            cp_async_commit();
            cp_async_wait<0>();
        }
        __syncthreads();
    };
    if (!OUT || pc.len == 0) enter();
    float decay = 1.f;
    for (int t0 = 0; t0 < pc.len; t0 += kC) {
        const int n = min(kC, pc.len - t0);
        const long long row = pc.row + t0;
        if (t0) __syncthreads();
        if (OUT) load_rows<DK>(Q, QS, (const float*)x.q + row * sh.qs + hk * sh.dk, sh.qs, n, sh.dk);
        load_rows<DK>(K, QS, (const float*)x.k + row * sh.ks + hk * sh.dk, sh.ks, n, sh.dk);
        load_rows<kTile>(V, kVS, (const float*)x.v + row * sh.vs + (long long)h * sh.dv + c0, sh.vs, n, cols);
        cp_async_commit();
        if (threadIdx.x < 32) chunk_exponents(sh, x.g, h, (int)row, n, ex);
        cp_async_wait<0>();
        __syncthreads();
        const Exponent last = ex[kC - 1];
        const float chunk = decay_of(last);
        decay *= chunk;
        if constexpr (OUT) {
            float o[4][4] = {}, a[4][4] = {};
            if (p.wc < 2 * p.wr + 2) mm_nt<4, true>(a, Q, QS, K, QS, sh.dk, p);
            if (t0 == 0) enter();
            if (live) mm_nn<4>(o, Q, QS, S, kVS, sh.dk, p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const Exponent e = ex[p.r0 + 8 * i];
                const float w = weight_of(e);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    o[i][j] *= w;
                    const int t = spread(p, j);
                    a[i][j] = t <= p.r0 + 8 * i ? a[i][j] * decay_between(e, ex[t]) : 0.f;
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) Q[(p.r0 + 8 * i) * kVS + spread(p, j)] = a[i][j];
            __syncthreads();
            if (live) {
                mm_nn<4>(o, Q, kVS, V, kVS, 32 * p.wr + 32, p);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = p.r0 + 8 * i;
                    if (r < n && c < cols) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[i][j] *= sh.scale;
                        store_vec<float, 4>((float*)x.y + ((size_t)(row + r) * sh.H + h) * sh.dv + c0 + c, o[i]);
                    }
                }
            }
            __syncthreads();
        }
        if (t0 + kC < pc.len || !OUT || last_state) {  // S = e^{G_C} S + sum_t k_t (e^{G_C - G_t} v_t)^T
#pragma unroll
            for (int i = threadIdx.x; i < kC * (kTile / 4); i += kThr) {
                const int r = i / (kTile / 4);
                float4* v = reinterpret_cast<float4*>(V + r * kVS + (i % (kTile / 4)) * 4);
                const float w = decay_between(last, ex[r]);
                float4 z = *v;
                z.x *= w; z.y *= w; z.z *= w; z.w *= w;
                *v = z;
            }
            __syncthreads();
            if (live) {
                float s[R][4];
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float4 z = *reinterpret_cast<const float4*>(S + (srow + i) * kVS + c);
                    s[i][0] = z.x * chunk; s[i][1] = z.y * chunk; s[i][2] = z.z * chunk; s[i][3] = z.w * chunk;
                }
                mm_tn<R>(s, K, QS, V, n, p);
#pragma unroll
                for (int i = 0; i < R; ++i)
                    *reinterpret_cast<float4*>(S + (srow + i) * kVS + c) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
            }
        }
    }
    cp_async_wait<0>();
    __syncthreads();
    float* s_out = !OUT ? st_loc + state_at
                   : last_state ? x.st + ((size_t)pc.seq * sh.H + h) * sh.dk * sh.dv : nullptr;
    if (s_out)
        for (int i = threadIdx.x; i < DK * (kTile / 4); i += kThr) {
            const int r = i / (kTile / 4), k = (i % (kTile / 4)) * 4;
            if (r < sh.dk && k < cols)
                *reinterpret_cast<float4*>(s_out + (size_t)r * sh.dv + c0 + k) = *reinterpret_cast<const float4*>(S + r * kVS + k);
        }
    if (!OUT && threadIdx.x == 0 && c0 == 0) piece_decay[(size_t)id * sh.H + h] = decay;
}

// ---- gradient -------------------------------------------------------------------------------------
struct GradOut {
    void *dq, *dk, *dv;      // dq, dk: the inputs' type, or fp32 per value head where heads share keys
    float* dg;               // [rows][H], or one sum per piece [pieces][H] with head_decay
    int partial;             // dq, dk are the fp32 per-head partials
};

template <int DK>
constexpr size_t local_smem() {
    return (size_t)(kC * row_stride(DK) + kC * kVS) * 4 + kC * sizeof(Exponent);
}

// Chunk-local states from zero.  One block per (chunk, head, 64 columns); blockIdx.z 0: sum_j e^{G_C - G_j}
// k_j v_j^T and the chunk's decay, 1: scale sum_i e^{G_i} q_i dy_i^T.
template <int DK>
__global__ void __launch_bounds__(kThr, 3)
simt_local_states_kernel(Shape sh, PackedPlan plan, Tensors x, float* __restrict__ S, float* __restrict__ dS,
                         float* __restrict__ decay, unsigned* status) {
    if (!sh.packed && blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
    extern __shared__ __align__(16) float sm[];
    constexpr int QS = row_stride(DK), R = DK / 16;
    float* A = sm;
    float* B = A + kC * QS;
    Exponent* ex = reinterpret_cast<Exponent*>(B + kC * kVS);
    Piece pc;
    int id;
    if (!get_piece(sh, plan, blockIdx.x, pc, id)) return;
    launch_dependents();
    const bool grad = blockIdx.z == 1;
    const int tiles = (sh.dv + kTile - 1) / kTile;
    const int h = blockIdx.y / tiles, c0 = (blockIdx.y - h * tiles) * kTile;
    const int hk = key_head(sh, h), cols = min(kTile, sh.dv - c0);
    const Place p = place();
    const int c = 4 * p.c4;
    const long long row = pc.row;
    if (pc.len > 0) {
        load_rows<DK>(A, QS, (grad ? (const float*)x.q + row * sh.qs : (const float*)x.k + row * sh.ks) + hk * sh.dk,
                      grad ? sh.qs : sh.ks, pc.len, sh.dk);
        load_rows<kTile>(B, kVS, (grad ? (const float*)x.dy + row * sh.ys : (const float*)x.v + row * sh.vs) + (long long)h * sh.dv + c0,
                         grad ? sh.ys : sh.vs, pc.len, cols);
    }
    cp_async_commit();
    if (threadIdx.x < 32) chunk_exponents(sh, x.g, h, pc.row, pc.len, ex);
    cp_async_wait<0>();
    __syncthreads();
    const Exponent last = ex[kC - 1];
    if (threadIdx.x == 0 && c0 == 0 && !grad) decay[(size_t)id * sh.H + h] = decay_of(last);
    for (int i = threadIdx.x; i < pc.len * (kTile / 4); i += kThr) {
        const int r = i / (kTile / 4);
        float4* v = reinterpret_cast<float4*>(B + r * kVS + (i % (kTile / 4)) * 4);
        const float w = grad ? sh.scale * weight_of(ex[r]) : decay_between(last, ex[r]);
        float4 z = *v;
        z.x *= w; z.y *= w; z.z *= w; z.w *= w;
        *v = z;
    }
    __syncthreads();
    if (c >= cols) return;
    float s[R][4] = {};
    mm_tn<R>(s, A, QS, B, pc.len, p);
    const int srow = R * (8 * p.wr + ((threadIdx.x & 31) >> 2));
    float* out = (grad ? dS : S) + ((size_t)id * sh.H + h) * sh.dk * sh.dv + c0 + c;
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (srow + i < sh.dk)
            *reinterpret_cast<float4*>(out + (size_t)(srow + i) * sh.dv) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
}

// P and its transpose over v and dy, M over A in the end.
template <int DK>
constexpr size_t grad_smem() {
    return (size_t)(2 * kC * row_stride(DK) + 2 * kC * kVS + DK * kVS + kC * kVS) * 4 + kC * sizeof(Exponent) + (2 * 4 + 8) * kC * 4 + 64;
}

// Gradients of one chunk and head, given the state entering it (S) and the gradient of the state leaving
// it (dS).  With w_ij = scale e^{G_i - G_j}, A = w q k^T, P = w dy v^T and M_ij = w_ij (q_i . k_j)(dy_i . v_j):
//   dq = scale e^{G_i} S dy_i + P k,  dk = e^{G_C - G_j} dS v_j + P^T q,  dv = e^{G_C - G_j} dS^T k_j + A^T dy,
//   dg_t = sum_{i >= t > j} M_ij + sum_{i >= t} q_i . (first part of dq_i) + sum_{j < t} k_j . (first part of dk_j)
//          + e^{G_C} <dS, S>.
// dg is a sum of the pairs that each g_t lies between: nothing is subtracted, where the shorter form
// (a reverse running sum of q . dq - k . dk) would cancel what lies on one side only.
template <int DK>
__global__ void __launch_bounds__(kThr, DK == 64 ? 2 : 1)
simt_grad_kernel(Shape sh, PackedPlan plan, Tensors x, const float* S_in, const float* dS_out, GradOut out) {
    extern __shared__ __align__(16) float sm[];
    constexpr int QS = row_stride(DK), NJ = DK / 16;
    float* Q = sm;
    float* K = Q + kC * QS;
    float* V = K + kC * QS;
    float* Y = V + kC * kVS;
    float* S = Y + kC * kVS;
    float* A = S + DK * kVS;
    Exponent* ex = reinterpret_cast<Exponent*>(A + kC * kVS);
    float* inq = reinterpret_cast<float*>(ex + kC);  // [4][kC]: by column block
    float* outk = inq + 4 * kC;                      // [4][kC]
    float* col = outk + 4 * kC;                      // [8][kC]: by warp
    float* red = col + 8 * kC;                       // [8], and two sums
    Piece pc;
    int id;
    if (!get_piece(sh, plan, blockIdx.x, pc, id)) return wait_for_primary();
    const int n = pc.len, h = blockIdx.y, hk = key_head(sh, h), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (n == 0) {
        wait_for_primary();  // no launch ends before those it overlaps
        if (sh.head_decay && threadIdx.x == 0) out.dg[(size_t)id * sh.H + h] = 0.f;
        return;
    }
    const Place p = place();
    const int c = 4 * p.c4, ck = NJ * p.c4;
    const long long row = pc.row;
    const size_t state_at = ((size_t)id * sh.H + h) * sh.dk * sh.dv;
    auto load_tile = [&](int c0) {
        const int cols = min(kTile, sh.dv - c0);
        if (c0 == 0) wait_for_primary();
        load_rows<kTile>(V, kVS, (const float*)x.v + row * sh.vs + (long long)h * sh.dv + c0, sh.vs, n, cols);
        load_rows<kTile>(Y, kVS, (const float*)x.dy + row * sh.ys + (long long)h * sh.dv + c0, sh.ys, n, cols);
        load_state<DK>(S, S_in + state_at + c0, sh.dk, sh.dv, cols);
        cp_async_commit();
    };
    load_rows<DK>(Q, QS, (const float*)x.q + row * sh.qs + hk * sh.dk, sh.qs, n, sh.dk);
    load_rows<DK>(K, QS, (const float*)x.k + row * sh.ks + hk * sh.dk, sh.ks, n, sh.dk);
    load_tile(0);
    if (threadIdx.x < 32) chunk_exponents(sh, x.g, h, pc.row, n, ex);
    cp_async_wait<0>();
    __syncthreads();
    const Exponent last = ex[kC - 1];
    const bool lower = p.wc < 2 * p.wr + 2;  // this warp's part of a token x token tile holds pairs j <= i
    {
        float a[4][4] = {};
        if (lower) mm_nt<4, true>(a, Q, QS, K, QS, sh.dk, p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = p.r0 + 8 * i;
            const Exponent e = ex[r];
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // transposed: its products run over i
                const int t = spread(p, j);
                A[t * kVS + r] = t <= r ? a[i][j] * sh.scale * decay_between(e, ex[t]) : 0.f;
            }
        }
    }
    float X[4][4] = {}, dq[4][NJ] = {}, dk[4][NJ] = {};
    const float root = root_decay_of(last);
    float dot = 0.f;  // e^{G_C} <dS, S>
    const bool klive = 4 * NJ * p.wc < sh.dk;  // this warp's columns of dq and dk
    for (int c0 = 0; c0 < sh.dv; c0 += kTile) {
        const int cols = min(kTile, sh.dv - c0);
        if (c0) {
            __syncthreads();
            load_tile(c0);
            cp_async_wait<0>();
            __syncthreads();
        }
        if (lower) mm_nt<4, true>(X, Y, kVS, V, kVS, cols, p);
        if (klive) mm_nt<NJ, false>(dq, Y, kVS, S, kVS, cols, p);
        __syncthreads();
        for (int i = threadIdx.x; i < DK * (kTile / 4); i += kThr) {
            const int r = i / (kTile / 4), k = (i % (kTile / 4)) * 4;
            float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < sh.dk && k < cols) d = __ldcg(reinterpret_cast<const float4*>(dS_out + state_at + (size_t)r * sh.dv + c0 + k));
            float4* s = reinterpret_cast<float4*>(S + r * kVS + k);
            const float4 z = *s;
            dot = fmaf(root * d.x, root * z.x, fmaf(root * d.y, root * z.y, fmaf(root * d.z, root * z.z, fmaf(root * d.w, root * z.w, dot))));
            *s = d;
        }
        __syncthreads();
        if (klive) mm_nt<NJ, false>(dk, V, kVS, S, kVS, cols, p);
        if (16 * p.wc < cols) {
            float dv[4][4] = {};
            mm_nn<4>(dv, K, QS, S, kVS, sh.dk, p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float w = decay_between(last, ex[p.r0 + 8 * i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) dv[i][j] *= w;
            }
            mm_nn<4>(dv, A + 32 * p.wr, kVS, Y + 32 * p.wr * kVS, kVS, kC - 32 * p.wr, p);  // i >= j
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (p.r0 + 8 * i < n && c < cols)
                    store_vec<float, 4>((float*)out.dv + ((size_t)(row + p.r0 + 8 * i) * sh.H + h) * sh.dv + c0 + c, dv[i]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // P over v, its transpose over dy, M over A
        const int r = p.r0 + 8 * i;
        const Exponent e = ex[r];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = spread(p, j);
            const bool in = t <= r;
            const float m = in ? A[t * kVS + r] * X[i][j] : 0.f, z = in ? X[i][j] * sh.scale * decay_between(e, ex[t]) : 0.f;
            X[i][j] = m;
            V[r * kVS + t] = z;
            Y[t * kVS + r] = z;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) A[(p.r0 + 8 * i) * kVS + spread(p, j)] = X[i][j];
    // the parts through the states, and their products with q and k
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = p.r0 + 8 * i;
        const float wq = sh.scale * weight_of(ex[r]), wk = decay_between(last, ex[r]);
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            dq[i][j] *= wq;
            dk[i][j] *= wk;
            a = fmaf(dq[i][j], Q[r * QS + ck + j], a);
            b = fmaf(dk[i][j], K[r * QS + ck + j], b);
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if ((lane & 3) == 0) {
            inq[p.wc * kC + r] = a;
            outk[p.wc * kC + r] = b;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) red[warp] = dot;
    __syncthreads();
    if (klive) {
        mm_nn<NJ>(dq, V, kVS, K, QS, 32 * p.wr + 32, p);
        mm_nn<NJ>(dk, Y + 32 * p.wr, kVS, Q + 32 * p.wr * QS, QS, kC - 32 * p.wr, p);
    }
    {
        // sum_{i >= t > j} M_ij: what lies left of column t in each row, summed over the rows from t on
        float s0 = 0.f, s1 = 0.f;  // columns 2 lane, 2 lane + 1
        for (int i = warp; i < n; i += kThr / 32) {
            const float2 m = *reinterpret_cast<const float2*>(A + i * kVS + 2 * lane);
            float s = m.x + m.y;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float v = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += v;
            }
            float before = __shfl_up_sync(0xffffffffu, s, 1);
            if (lane == 0) before = 0.f;
            if (2 * lane <= i) s0 += before;
            if (2 * lane + 1 <= i) s1 += before + m.x;
        }
        *reinterpret_cast<float2*>(col + warp * kC + 2 * lane) = make_float2(s0, s1);
    }
    __syncthreads();
    if (warp < 2) {
        const int t = 32 * warp + lane;
        float a = 0.f, iq = 0.f, ok = 0.f;
        for (int i = 0; i < 8; ++i) a += col[i * kC + t];
        for (int i = 0; i < 4; ++i) {
            iq += inq[i * kC + t];
            ok += outk[i * kC + t];
        }
        // the sums of the other half of the tokens: leaving before t, entering behind it
        float other = 0.f;
        for (int i = 0; i < 4; ++i) other += warp == 0 ? inq[i * kC + 32 + lane] : outk[i * kC + lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) other += __shfl_xor_sync(0xffffffffu, other, o);
        float sq = iq, sk = __shfl_up_sync(0xffffffffu, ok, 1);  // from this token on; before it
        if (lane == 0) sk = 0.f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float u = __shfl_down_sync(0xffffffffu, sq, o), v = __shfl_up_sync(0xffffffffu, sk, o);
            if (lane + o < 32) sq += u;
            if (lane >= o) sk += v;
        }
        float d = 0.f;
        for (int i = 0; i < 8; ++i) d += red[i];
        a += sq + sk + other;
        a += d;
        if (t >= n) a = 0.f;
        if (!sh.head_decay) {
            if (t < n) out.dg[(size_t)(row + t) * sh.H + h] = a;
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
            if (lane == 0) red[8 + warp] = a;
        }
    }
    if (klive && ck < sh.dk) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = p.r0 + 8 * i;
            if (r >= n) continue;
            const size_t at = out.partial ? ((size_t)(row + r) * sh.H + h) * sh.dk + ck : ((size_t)(row + r) * sh.Hk + hk) * sh.dk + ck;
#pragma unroll
            for (int j = 0; j < NJ; j += 4) {
                *reinterpret_cast<float4*>((float*)out.dq + at + j) = make_float4(dq[i][j], dq[i][j + 1], dq[i][j + 2], dq[i][j + 3]);
                *reinterpret_cast<float4*>((float*)out.dk + at + j) = make_float4(dk[i][j], dk[i][j + 1], dk[i][j + 2], dk[i][j + 3]);
            }
        }
    }
    if (sh.head_decay) {
        __syncthreads();
        if (threadIdx.x == 0) out.dg[(size_t)id * sh.H + h] = red[8] + red[9];
    }
}

}  // namespace la
}  // namespace fv
