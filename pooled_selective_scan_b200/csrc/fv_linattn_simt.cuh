// fv_linattn_simt.cuh -- linear attention on fp32 FMAs: the fp32 forward and gradient.
#pragma once

#include "fv_linattn.cuh"

namespace fv {
namespace la {

constexpr int kC = 64;        // tokens per chunk
constexpr int kThr = 256;
constexpr int kPS = kC + 4;   // row stride of a token x token tile

__host__ __device__ constexpr int row_stride(int d) { return d + 4; }

// Rows [0, kC) of columns [c0, c0 + W) of a token-major tensor into sm (row stride `stride`); zeros behind
// the piece's tokens and behind `cols`.
template <typename T>
__device__ __forceinline__ void load_rows(float* sm, int stride, int W, const T* src, long long token_stride, int n,
                                          int cols) {
    const int per = W / 4;
    for (int i = threadIdx.x; i < kC * per; i += kThr) {
        const int r = i / per, c = (i - r * per) * 4;
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (r < n && c < cols) load_vec<T, 4, false>(src + (long long)r * token_stride + c, x);
        *reinterpret_cast<float4*>(sm + r * stride + c) = make_float4(x[0], x[1], x[2], x[3]);
    }
}

// acc[4][4] += A rows (ty + 16 i) . B rows (tx + 16 j) over K columns (both token-major).
__device__ __forceinline__ void mm_nt(float (&acc)[4][4], const float* A, int as, const float* B, int bs, int K, int ty,
                                      int tx) {
    for (int k = 0; k < K; k += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(A + (ty + 16 * i) * as + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * bs + k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, acc[i][j]))));
    }
}
// acc[4][NC] += A[rows ty + 16 i][K] * B[K][columns c .. c + NC)
template <int NC>
__device__ __forceinline__ void mm_nn(float (&acc)[4][NC], const float* A, int as, const float* B, int bs, int K, int ty,
                                      int c) {
    for (int k = 0; k < K; k += 4) {
        float4 a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(A + (ty + 16 * i) * as + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            float b[NC];
#pragma unroll
            for (int j = 0; j < NC; j += 4) {
                const float4 v = *reinterpret_cast<const float4*>(B + (k + kk) * bs + c + j);
                b[j] = v.x; b[j + 1] = v.y; b[j + 2] = v.z; b[j + 3] = v.w;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = kk == 0 ? a[i].x : kk == 1 ? a[i].y : kk == 2 ? a[i].z : a[i].w;
#pragma unroll
                for (int j = 0; j < NC; ++j) acc[i][j] = fmaf(x, b[j], acc[i][j]);
            }
        }
    }
}
// acc[NR][NC] += sum over tokens t of A[t][r .. r + NR) * B[t][c .. c + NC)
template <int NR, int NC>
__device__ __forceinline__ void mm_tn(float (&acc)[NR][NC], const float* A, int as, const float* B, int bs, int K, int r,
                                      int c) {
#pragma unroll 4
    for (int t = 0; t < K; ++t) {
        float a[NR], b[NC];
#pragma unroll
        for (int i = 0; i < NR; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(A + t * as + r + i);
            a[i] = v.x; a[i + 1] = v.y; a[i + 2] = v.z; a[i + 3] = v.w;
        }
#pragma unroll
        for (int j = 0; j < NC; j += 4) {
            const float4 v = *reinterpret_cast<const float4*>(B + t * bs + c + j);
            b[j] = v.x; b[j + 1] = v.y; b[j + 2] = v.z; b[j + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int j = 0; j < NC; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
}

// DK: dk rounded up to 64 or 128.
template <int DK>
constexpr size_t fwd_smem() {
    return (size_t)(2 * kC * row_stride(DK) + 2 * kC * row_stride(kTile) + DK * row_stride(kTile) + kC * kPS) * 4 +
           kC * sizeof(Exponent) + 64;
}

// One piece, head and 64 columns of v: walks the piece's chunks with the state in shared memory.
// OUT: writes y (and, behind the sequence's last piece, the final state).  Without it: the piece's own
// state from zero into st_loc and its decay into piece_decay.
template <typename T, int DK, bool OUT>
__global__ void __launch_bounds__(kThr) simt_kernel(Shape sh, PackedPlan plan, Tensors x, const float* __restrict__ start,
                                                    float* __restrict__ st_loc, float* __restrict__ piece_decay) {
    extern __shared__ __align__(16) float sm[];
    constexpr int QS = row_stride(DK), VS = row_stride(kTile);
    float* Q = sm;
    float* K = Q + kC * QS;
    float* V = K + kC * QS;
    float* VW = V + kC * VS;  // v weighted for the state
    float* S = VW + kC * VS;
    float* P = S + DK * VS;
    Exponent* ex = reinterpret_cast<Exponent*>(P + kC * kPS);
    Piece pc;
    if (!get_piece(sh, plan, blockIdx.x, pc)) return;
    // a piece's own state is needed where another follows, or where its sequence's final state is asked for;
    // a sequence of one piece carries its state alone
    if (!OUT && (pc.flags == 3 || ((pc.flags & 2) && !x.st))) return;
    const int tiles = (sh.dv + kTile - 1) / kTile;
    const int h = blockIdx.y / tiles, c0 = (blockIdx.y - h * tiles) * kTile;
    const int hk = key_head(sh, h), cols = min(kTile, sh.dv - c0);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const size_t state_at = ((size_t)blockIdx.x * sh.H + h) * sh.dk * sh.dv;
    const float* s_in = !OUT ? nullptr : pc.flags != 3 ? start + state_at
                        : x.s0 ? x.s0 + ((size_t)pc.seq * sh.H + h) * sh.dk * sh.dv : nullptr;
    for (int i = threadIdx.x; i < DK * kTile; i += kThr) {
        const int r = i / kTile, c = i - r * kTile;
        S[r * VS + c] = s_in && r < sh.dk && c < cols ? s_in[(size_t)r * sh.dv + c0 + c] : 0.f;
    }
    double total = 0.0;
    for (int t0 = 0; t0 < pc.len; t0 += kC) {
        const int n = min(kC, pc.len - t0), row = pc.row + t0;
        __syncthreads();
        if (OUT) load_rows<T>(Q, QS, DK, (const T*)x.q + (long long)row * sh.qs + hk * sh.dk, sh.qs, n, sh.dk);
        load_rows<T>(K, QS, DK, (const T*)x.k + (long long)row * sh.ks + hk * sh.dk, sh.ks, n, sh.dk);
        load_rows<T>(V, VS, kTile, (const T*)x.v + (long long)row * sh.vs + (long long)h * sh.dv + c0, sh.vs, n, cols);
        if (threadIdx.x < 32) {
            const double t = warp_exponents<kC>(sh, x.g, h, row, n, ex);
            if (!OUT) total += t;
        }
        __syncthreads();
        const Exponent last = ex[kC - 1];
        for (int i = threadIdx.x; i < kC * kTile; i += kThr) {
            const int r = i / kTile, c = i - r * kTile;
            VW[r * VS + c] = r < n ? V[r * VS + c] * decay_between(last, ex[r]) : 0.f;
        }
        if constexpr (OUT) {
            float p[4][4] = {};
            mm_nt(p, Q, QS, K, QS, DK, ty, tx);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int a = ty + 16 * i, b = tx + 16 * j;
                    P[a * kPS + b] = b <= a ? p[i][j] * decay_between(ex[a], ex[b]) : 0.f;
                }
            float o[4][4] = {};
            mm_nn<4>(o, Q, QS, S, VS, DK, ty, tx * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float w = ex2_approx(ex[ty + 16 * i].hi + ex[ty + 16 * i].lo);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][j] *= w;
            }
            __syncthreads();
            mm_nn<4>(o, P, kPS, V, VS, kC, ty, tx * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = ty + 16 * i;
                if (r < n && tx * 4 < cols) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[i][j] *= sh.scale;
                    store_vec<T, 4>((T*)x.y + ((size_t)(row + r) * sh.H + h) * sh.dv + c0 + tx * 4, o[i]);
                }
            }
        } else {
            __syncthreads();
        }
        // S = e^{G_C} S + sum_t k_t (weighted v_t)^T; thread: DK / 16 rows x 4 columns
        const float w = ex2_approx(last.hi + last.lo);
        constexpr int kR = DK / 16;
        float s[kR][4];
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = S[(ty * kR + i) * VS + tx * 4 + j] * w;
        mm_tn<kR, 4>(s, K, QS, VW, VS, n, ty * kR, tx * 4);
#pragma unroll
        for (int i = 0; i < kR; ++i)
            *reinterpret_cast<float4*>(S + (ty * kR + i) * VS + tx * 4) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
    }
    __syncthreads();
    float* s_out = !OUT ? st_loc + state_at
                   : (x.st && pc.flags == 3) ? x.st + ((size_t)pc.seq * sh.H + h) * sh.dk * sh.dv : nullptr;
    if (s_out)
        for (int i = threadIdx.x; i < DK * kTile; i += kThr) {
            const int r = i / kTile, c = i - r * kTile;
            if (r < sh.dk && c < cols) s_out[(size_t)r * sh.dv + c0 + c] = S[r * VS + c];
        }
    if (!OUT && threadIdx.x == 0 && c0 == 0) piece_decay[(size_t)blockIdx.x * sh.H + h] = exp2f((float)total);
}

// ---- gradient -------------------------------------------------------------------------------------
// acc[4][NJ] (rows ty + 16 i, columns tx + 16 j) += A[rows][K] . B[columns][K]
template <int NJ>
__device__ __forceinline__ void mm_nt_cols(float (&acc)[4][NJ], const float* A, int as, const float* B, int bs, int K,
                                           int ty, int tx) {
#pragma unroll 2
    for (int k = 0; k < K; k += 4) {
        float4 a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(A + (ty + 16 * i) * as + k);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const float4 b = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * bs + k);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[i][j] = fmaf(a[i].x, b.x, fmaf(a[i].y, b.y, fmaf(a[i].z, b.z, fmaf(a[i].w, b.w, acc[i][j]))));
        }
    }
}
// acc[4][NJ] (columns tx + 16 j) += A (AT ? A[t][ty + 16 i] : A[ty + 16 i][t]) B[t][column], t < K
template <int NJ, bool AT>
__device__ __forceinline__ void mm_cols(float (&acc)[4][NJ], const float* A, int as, const float* B, int bs, int K, int ty,
                                        int tx) {
#pragma unroll 4
    for (int t = 0; t < K; ++t) {
        float a[4], b[NJ];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = AT ? A[t * as + ty + 16 * i] : A[(ty + 16 * i) * as + t];
#pragma unroll
        for (int j = 0; j < NJ; ++j) b[j] = B[t * bs + tx + 16 * j];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
}

struct GradOut {
    void *dq, *dk, *dv;      // dq, dk: T, or fp32 per value head where heads share keys
    float* dg;               // [rows][H], or one sum per piece [pieces][H] with head_decay
    int partial;             // dq, dk are the fp32 per-head partials
};

// Chunk-local states from zero: sum_j e^{G_C - G_j} k_j v_j^T and scale sum_i e^{G_i} q_i dy_i^T, and the
// chunk's decay.  One block per (chunk, head, 64 columns).
template <typename T, int DK>
__global__ void __launch_bounds__(kThr) simt_local_states_kernel(Shape sh, PackedPlan plan, Tensors x, float* __restrict__ S,
                                                                 float* __restrict__ dS, float* __restrict__ decay) {
    extern __shared__ __align__(16) float sm[];
    constexpr int QS = row_stride(DK), VS = row_stride(kTile), kR = DK / 16;
    float* A = sm;
    float* B = A + kC * QS;
    Exponent* ex = reinterpret_cast<Exponent*>(B + kC * VS);
    Piece pc;
    if (!get_piece(sh, plan, blockIdx.x, pc)) return;
    const int tiles = (sh.dv + kTile - 1) / kTile;
    const int h = blockIdx.y / tiles, c0 = (blockIdx.y - h * tiles) * kTile;
    const int hk = key_head(sh, h), cols = min(kTile, sh.dv - c0);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    if (threadIdx.x < 32) {
        const double t = warp_exponents<kC>(sh, x.g, h, pc.row, pc.len, ex);
        if (threadIdx.x == 0 && c0 == 0) decay[(size_t)blockIdx.x * sh.H + h] = exp2f((float)t);
    }
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        __syncthreads();
        if (pass == 0) {
            load_rows<T>(A, QS, DK, (const T*)x.k + (long long)pc.row * sh.ks + hk * sh.dk, sh.ks, pc.len, sh.dk);
            load_rows<T>(B, VS, kTile, (const T*)x.v + (long long)pc.row * sh.vs + (long long)h * sh.dv + c0, sh.vs, pc.len, cols);
        } else {
            load_rows<T>(A, QS, DK, (const T*)x.q + (long long)pc.row * sh.qs + hk * sh.dk, sh.qs, pc.len, sh.dk);
            load_rows<T>(B, VS, kTile, (const T*)x.dy + (long long)pc.row * sh.ys + (long long)h * sh.dv + c0, sh.ys, pc.len, cols);
        }
        __syncthreads();
        const Exponent last = ex[kC - 1];
        for (int i = threadIdx.x; i < kC * kTile; i += kThr) {
            const int r = i / kTile, c = i - r * kTile;
            B[r * VS + c] *= pass == 0 ? decay_between(last, ex[r]) : sh.scale * ex2_approx(ex[r].hi + ex[r].lo);
        }
        __syncthreads();
        float s[kR][4] = {};
        mm_tn<kR, 4>(s, A, QS, B, VS, pc.len, ty * kR, tx * 4);
        float* out = (pass == 0 ? S : dS) + ((size_t)blockIdx.x * sh.H + h) * sh.dk * sh.dv + c0;
        if (tx * 4 < cols)
#pragma unroll
            for (int i = 0; i < kR; ++i)
                if (ty * kR + i < sh.dk)
                    *reinterpret_cast<float4*>(out + (size_t)(ty * kR + i) * sh.dv + tx * 4) =
                        make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
    }
}

template <int DK>
constexpr size_t grad_smem() {
    return (size_t)(2 * kC * row_stride(DK) + 2 * kC * row_stride(kTile) + DK * row_stride(kTile) + 2 * kC * kPS) * 4 +
           kC * sizeof(Exponent) + (3 * kC + 16) * 4;
}

// Gradients of one chunk and head, given the state entering it (S) and the gradient of the state leaving
// it (dS).  With w_ij = scale e^{G_i - G_j}, A = w q k^T, P = w dy v^T and M_ij = w_ij (q_i . k_j)(dy_i . v_j):
//   dq = scale e^{G_i} S dy_i + P k,  dk = e^{G_C - G_j} dS v_j + P^T q,  dv = e^{G_C - G_j} dS^T k_j + A^T dy,
//   dg_t = sum_{i >= t > j} M_ij + sum_{i >= t} q_i . (first part of dq_i) + sum_{j < t} k_j . (first part of dk_j)
//          + e^{G_C} <dS, S>.
// dg is a sum of the pairs that each g_t lies between: nothing is subtracted, where the shorter form
// (a reverse running sum of q . dq - k . dk) would cancel what lies on one side only.
template <typename T, int DK>
__global__ void __launch_bounds__(kThr) simt_grad_kernel(Shape sh, PackedPlan plan, Tensors x, const float* __restrict__ S_in,
                                                         const float* __restrict__ dS_out, GradOut out) {
    extern __shared__ __align__(16) float sm[];
    constexpr int QS = row_stride(DK), VS = row_stride(kTile), NJ = DK / 16;
    float* Q = sm;
    float* K = Q + kC * QS;
    float* V = K + kC * QS;
    float* Y = V + kC * VS;
    float* S = Y + kC * VS;
    float* A = S + DK * VS;
    float* P = A + kC * kPS;
    Exponent* ex = reinterpret_cast<Exponent*>(P + kC * kPS);
    float* inq = reinterpret_cast<float*>(ex + kC);
    float* outk = inq + kC;
    float* dgs = outk + kC;
    float* red = dgs + kC;
    Piece pc;
    if (!get_piece(sh, plan, blockIdx.x, pc)) return;
    const int n = pc.len, h = blockIdx.y, hk = key_head(sh, h);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    if (n == 0) {
        if (sh.head_decay && threadIdx.x == 0) out.dg[(size_t)blockIdx.x * sh.H + h] = 0.f;
        return;
    }
    load_rows<T>(Q, QS, DK, (const T*)x.q + (long long)pc.row * sh.qs + hk * sh.dk, sh.qs, n, sh.dk);
    load_rows<T>(K, QS, DK, (const T*)x.k + (long long)pc.row * sh.ks + hk * sh.dk, sh.ks, n, sh.dk);
    if (threadIdx.x < 32) warp_exponents<kC>(sh, x.g, h, pc.row, n, ex);
    __syncthreads();
    const Exponent last = ex[kC - 1];
    {
        float a[4][4] = {};
        mm_nt(a, Q, QS, K, QS, DK, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = ty + 16 * i, c = tx + 16 * j;
                A[r * kPS + c] = c <= r ? a[i][j] * sh.scale * decay_between(ex[r], ex[c]) : 0.f;
            }
    }
    float X[4][4] = {}, dq[4][NJ] = {}, dk[4][NJ] = {};
    float dot = 0.f;
    const size_t state_at = ((size_t)blockIdx.x * sh.H + h) * sh.dk * sh.dv;
    for (int c0 = 0; c0 < sh.dv; c0 += kTile) {
        const int cols = min(kTile, sh.dv - c0);
        __syncthreads();
        load_rows<T>(V, VS, kTile, (const T*)x.v + (long long)pc.row * sh.vs + (long long)h * sh.dv + c0, sh.vs, n, cols);
        load_rows<T>(Y, VS, kTile, (const T*)x.dy + (long long)pc.row * sh.ys + (long long)h * sh.dv + c0, sh.ys, n, cols);
        for (int i = threadIdx.x; i < DK * kTile; i += kThr) {
            const int r = i / kTile, c = i - r * kTile;
            S[r * VS + c] = r < sh.dk && c < cols ? S_in[state_at + (size_t)r * sh.dv + c0 + c] : 0.f;
        }
        __syncthreads();
        mm_nt(X, Y, VS, V, VS, kTile, ty, tx);
        mm_nt_cols<NJ>(dq, Y, VS, S, VS, kTile, ty, tx);
        __syncthreads();
        for (int i = threadIdx.x; i < DK * kTile; i += kThr) {
            const int r = i / kTile, c = i - r * kTile;
            const float d = r < sh.dk && c < cols ? dS_out[state_at + (size_t)r * sh.dv + c0 + c] : 0.f;
            dot = fmaf(d, S[r * VS + c], dot);
            S[r * VS + c] = d;
        }
        __syncthreads();
        mm_nt_cols<NJ>(dk, V, VS, S, VS, kTile, ty, tx);
        float dv[4][4] = {};
        mm_cols<4, false>(dv, K, QS, S, VS, DK, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float w = decay_between(last, ex[ty + 16 * i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) dv[i][j] *= w;
        }
        mm_cols<4, true>(dv, A, kPS, Y, VS, kC, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 16 * i;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (r < n && tx + 16 * j < cols) {
                    const size_t at = ((size_t)(pc.row + r) * sh.H + h) * sh.dv + c0 + tx + 16 * j;
                    if constexpr (sizeof(T) == 4) ((float*)out.dv)[at] = dv[i][j];
                    else ((T*)out.dv)[at] = __float2bfloat16_rn(dv[i][j]);
                }
        }
    }
    __syncthreads();
    // M into V's tile, P into its own
    static_assert(row_stride(kTile) >= kPS, "M takes V's tile");
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = ty + 16 * i, c = tx + 16 * j;
            P[r * kPS + c] = c <= r ? X[i][j] * sh.scale * decay_between(ex[r], ex[c]) : 0.f;
            V[r * VS + c] = c <= r ? A[r * kPS + c] * X[i][j] : 0.f;
        }
    // the parts through the states, and their products with q and k
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
        const float wq = sh.scale * ex2_approx(ex[r].hi + ex[r].lo), wk = decay_between(last, ex[r]);
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            dq[i][j] *= wq;
            dk[i][j] *= wk;
            a = fmaf(dq[i][j], Q[r * QS + tx + 16 * j], a);
            b = fmaf(dk[i][j], K[r * QS + tx + 16 * j], b);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if (tx == 0) inq[r] = a, outk[r] = b;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = dot;
    __syncthreads();
    mm_cols<NJ, false>(dq, P, kPS, K, QS, kC, ty, tx);
    mm_cols<NJ, true>(dk, P, kPS, Q, QS, kC, ty, tx);
    if (threadIdx.x < kC) {  // row prefixes of M: what lies left of t
        float a = 0.f;
        for (int t = 0; t < kC; ++t) {
            const float m = V[threadIdx.x * VS + t];
            V[threadIdx.x * VS + t] = a;
            a += m;
        }
    }
    __syncthreads();
    if (threadIdx.x < kC) {
        const int t = threadIdx.x;
        float a = 0.f;
        for (int i = t; i < n; ++i) a += V[i * VS + t] + inq[i];
        for (int j = 0; j < t && j < n; ++j) a += outk[j];
        float d = 0.f;
        for (int i = 0; i < kThr / 32; ++i) d += red[i];
        a = fmaf(d, ex2_approx(last.hi + last.lo), a);
        dgs[t] = t < n ? a : 0.f;
        if (!sh.head_decay && t < n) out.dg[(size_t)(pc.row + t) * sh.H + h] = a;
    }
    __syncthreads();
    if (sh.head_decay && threadIdx.x == 0) {
        float a = 0.f;
        for (int t = 0; t < n; ++t) a += dgs[t];
        out.dg[(size_t)blockIdx.x * sh.H + h] = a;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int c = tx + 16 * j;
            if (r >= n || c >= sh.dk) continue;
            if (out.partial) {
                const size_t at = ((size_t)(pc.row + r) * sh.H + h) * sh.dk + c;
                ((float*)out.dq)[at] = dq[i][j];
                ((float*)out.dk)[at] = dk[i][j];
            } else {
                const size_t at = ((size_t)(pc.row + r) * sh.Hk + hk) * sh.dk + c;
                if constexpr (sizeof(T) == 4) {
                    ((float*)out.dq)[at] = dq[i][j];
                    ((float*)out.dk)[at] = dk[i][j];
                } else {
                    ((T*)out.dq)[at] = __float2bfloat16_rn(dq[i][j]);
                    ((T*)out.dk)[at] = __float2bfloat16_rn(dk[i][j]);
                }
            }
        }
    }
}

}  // namespace la
}  // namespace fv
