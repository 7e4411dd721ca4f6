// fv_linattn.cu -- linear attention with a decay for each head: C ABI, planning and launches, and the
// kernels around the chunk products (packed-sequence plan, joining of pieces, single-token step).
// Definitions, layouts and errors: fastvim_ssm.h.
#include <string.h>

#include <algorithm>

#include "fv_host.cuh"
#include "fv_linattn.cuh"
#include "fv_linattn_simt.cuh"
#include "fv_linattn_tc.cuh"
#include "fv_linattn_tc_grad.cuh"

namespace fv {
namespace la {
namespace {

// ---- packed sequences: pieces of at most L tokens ---------------------------------------------------
// control: [0] status (by the kernels' rules the first error stays), [1] pieces in use, [2], [3] the rows
// [lo, hi) that hold tokens, [4] pieces of sequences that are cut, whose numbers `cut` lists.  An offset list that falls, or leaves [0, T], leaves nothing to do.
__global__ void __launch_bounds__(1024) plan_kernel(const int* __restrict__ cu, int N, int T, int L, int most, int* control,
                                                    int* first_of, Piece* table, int* order, int* cut) {
    __shared__ int warp_sum[32];
    __shared__ int carry, bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) carry = 0, bad = 0;
    __syncthreads();
    for (int n = tid; n < N; n += 1024) {
        const int a = cu[n], b = cu[n + 1];
        if (a < 0 || b < a || b > T) bad = 1;
    }
    __syncthreads();
    const bool ok = bad == 0;
    for (int n0 = 0; n0 < N; n0 += 1024) {
        const int n = n0 + tid;
        int c = 0;
        if (ok && n < N) {
            const int len = cu[n + 1] - cu[n];
            c = len > 0 ? (len - 1) / L + 1 : 1;  // an empty sequence still passes its state on
        }
        int s = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        if (lane == 31) warp_sum[warp] = s;
        __syncthreads();
        if (warp == 0) {
            int w = warp_sum[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= o) w += u;
            }
            warp_sum[lane] = w;
        }
        __syncthreads();
        const int before = carry + s - c + (warp ? warp_sum[warp - 1] : 0);
        if (n < N) first_of[n] = before;
        __syncthreads();
        if (tid == 0) carry += warp_sum[31];
        __syncthreads();
    }
    const int count = min(carry, most);
    if (tid == 0) {
        first_of[N] = count;
        control[0] = ok ? 0 : (int)kStatusIndex;
        control[1] = count;
        control[2] = ok && N > 0 ? cu[0] : 0;
        control[3] = ok && N > 0 ? cu[N] : 0;
        control[4] = 0;
    }
    __syncthreads();
    for (int i = tid; i < count; i += 1024) {
        int lo = 0, hi = N;  // the last sequence whose first piece is <= i
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first_of[mid] <= i) lo = mid;
            else hi = mid;
        }
        const int c = i - first_of[lo], len = cu[lo + 1] - cu[lo], at = c * L;
        Piece p;
        p.seq = lo;
        p.row = cu[lo] + at;
        p.len = min(L, len - at);
        p.flags = (c == 0 ? 1 : 0) | (len - at <= L ? 2 : 0);
        table[i] = p;
        if (cut && p.flags != 3) cut[atomicAdd(control + 4, 1)] = i;
    }
    if (!order) return;
    // By falling length, in 256 steps: a long piece that starts last would end last by its whole length.
    // Which of two of a step comes first does not change a result.
    __shared__ int bucket[257];
    for (int i = tid; i < 257; i += 1024) bucket[i] = 0;
    __syncthreads();
    auto step_of = [&](int len) { return 255 - (int)((long long)len * 255 / L); };
    for (int i = tid; i < count; i += 1024) atomicAdd(&bucket[step_of(table[i].len) + 1], 1);
    __syncthreads();
    if (warp == 0) {
        int base = 0;
        for (int k = lane; k < 256; k += 32) {
            int s = bucket[k + 1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += u;
            }
            const int total = __shfl_sync(0xffffffffu, s, 31);
            bucket[k + 1] = base + s;
            base += total;
        }
    }
    __syncthreads();
    for (int i = tid; i < count; i += 1024) order[atomicAdd(&bucket[step_of(table[i].len)], 1)] = i;
}

// ---- joining pieces ---------------------------------------------------------------------------------
// Turns the pieces' own states into the states entering them, in place: per element
// run = start; for each piece: (st, run) = (run, decay run + st).  REVERSE walks from the last piece with
// the gradient of the final state.  `end`: where the state behind the last piece goes (the final state, or
// the gradient of the first one); without it the last piece's own state is not read.  Bound by its
// traffic (each state read and written once); eight pieces' loads are in flight at a time.  Both directions of
// 8 x 32 chunks x 12 heads of 64 x 64 (201 MB, some of it still in L2): 29 us.
template <bool REVERSE>
__device__ __forceinline__ void join(const Shape& sh, const int* first_of, float* st, const float* decay, const float* start,
                                     float* end, int seq, int h, int at) {
    const int p0 = sh.packed ? first_of[seq] : seq * sh.per_seq;
    const int p1 = sh.packed ? first_of[seq + 1] : p0 + sh.per_seq;
    const size_t size = (size_t)sh.dk * sh.dv, own = ((size_t)seq * sh.H + h) * size + at;
    float4 run = start ? *reinterpret_cast<const float4*>(start + own) : make_float4(0.f, 0.f, 0.f, 0.f);
    const int n = p1 - p0;
    constexpr int kU = 8;
    for (int c0 = 0; c0 < n; c0 += kU) {
        float4 v[kU];
        float d[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int c = c0 + u;
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            d[u] = 0.f;
            if (c < n && (end || c + 1 < n)) {
                const size_t p = (size_t)(REVERSE ? p1 - 1 - c : p0 + c) * sh.H + h;
                v[u] = *reinterpret_cast<const float4*>(st + p * size + at);
                d[u] = decay[p];
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int c = c0 + u;
            if (c >= n) break;
            const size_t p = (size_t)(REVERSE ? p1 - 1 - c : p0 + c) * sh.H + h;
            *reinterpret_cast<float4*>(st + p * size + at) = run;
            run = make_float4(fmaf(d[u], run.x, v[u].x), fmaf(d[u], run.y, v[u].y), fmaf(d[u], run.z, v[u].z),
                              fmaf(d[u], run.w, v[u].w));
        }
    }
    if (end) *reinterpret_cast<float4*>(end + own) = run;
}

// Every launch waits for the one that it overlaps, one that has nothing to do too: the kernel behind it may begin
// as soon as it has ended, and would else meet a launch that still runs (and the next call its workspace in use).
// One thread that waits keeps a launch from ending.
__device__ __forceinline__ bool first_block() { return blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0; }

__global__ void __launch_bounds__(256) join_kernel(Shape sh, const int* first_of, const int* control, float* st,
                                                   const float* decay, const float* start, float* end) {
    const int at = (blockIdx.y * 256 + threadIdx.x) * 4;
    const int seq = blockIdx.x / sh.H, h = blockIdx.x - seq * sh.H;
    const int n = !sh.packed ? sh.per_seq : control[1] == 0 ? 0 : first_of[seq + 1] - first_of[seq];
    const bool walks = at < sh.dk * sh.dv && n > 1;  // one piece carries its state alone
    launch_dependents();
    if (walks || first_block()) wait_for_primary();
    if (walks) join<false>(sh, first_of, st, decay, start, end, seq, h, at);
}
__global__ void __launch_bounds__(256) join_grad_kernel(Shape sh, const int* first_of, const int* control, float* S, float* dS,
                                                        const float* decay, const float* s0, const float* ds, float* ds0) {
    const int at = (blockIdx.y * 256 + threadIdx.x) * 4;
    const int seq = blockIdx.x / sh.H, h = blockIdx.x - seq * sh.H;
    const bool walks = at < sh.dk * sh.dv && !(sh.packed && control[1] == 0);
    launch_dependents();
    if (walks || first_block()) wait_for_primary();
    if (!walks) return;
    if (blockIdx.z == 0) join<false>(sh, first_of, S, decay, s0, nullptr, seq, h, at);
    else join<true>(sh, first_of, dS, decay, ds, ds0, seq, h, at);
}

// ---- sums of the gradients ---------------------------------------------------------------------------
// out[row][hk][c] = sum over the value heads of key head hk of part[row][h][c], in head order.
template <typename T>
__global__ void __launch_bounds__(256) fold_heads_kernel(Shape sh, const int* control, const float* __restrict__ pq,
                                                         const float* __restrict__ pk, T* __restrict__ dq, T* __restrict__ dk,
                                                         long long rows) {
    const int per = sh.Hk * sh.dk / 4, rep = sh.H / sh.Hk;
    const long long lo = sh.packed ? control[2] : 0, hi = sh.packed ? control[3] : rows;
    const float* part = blockIdx.y ? pk : pq;
    T* out = blockIdx.y ? dk : dq;
    for (long long i = lo * per + (long long)blockIdx.x * 256 + threadIdx.x; i < hi * per; i += (long long)gridDim.x * 256) {
        const long long row = i / per;
        const int e = (int)(i - row * per) * 4, hk = e / sh.dk, c = e - hk * sh.dk;
        float a[4] = {0.f, 0.f, 0.f, 0.f};
        for (int r = 0; r < rep; ++r) {
            const float4 v = __ldcs(reinterpret_cast<const float4*>(part + ((size_t)row * sh.H + hk * rep + r) * sh.dk + c));
            a[0] += v.x; a[1] += v.y; a[2] += v.z; a[3] += v.w;
        }
        store_vec<T, 4>(out + ((size_t)row * sh.Hk + hk) * sh.dk + c, a);
    }
}
// dg[h] = sum over the pieces of their sums, in a fixed order.
__global__ void __launch_bounds__(256) fold_decay_kernel(Shape sh, const int* control, const float* __restrict__ part,
                                                         float* __restrict__ dg) {
    __shared__ float red[8];
    const int h = blockIdx.x, n = sh.packed ? control[1] : sh.pieces;
    float a = 0.f;
    for (int i = threadIdx.x; i < n; i += 256) a += part[(size_t)i * sh.H + h];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
        a = 0.f;
        for (int i = 0; i < 8; ++i) a += red[i];
        dg[h] = a;
    }
}

// ---- single tokens -------------------------------------------------------------------------------------
// One token of B sequences: S = e^g S + k v^T in place, y = scale S^T q.  The state's traffic (8 dk dv
// bytes a row and head) is the floor.  Block: 128 threads, one (row, head, 64 columns of v); a thread
// holds one float4 of every eighth state row, all loads in flight before the first use.  256 rows of 12 heads
// of 128 x 128: 67 us, 0.92 of a 6.53 TB/s copy.  Registers for 16 rows a thread where 8 or 4 do: 24.6 -> 26.7
// us at dk 64, 22.7 -> 36.8 us at dk 32.
struct StepParams {
    int B, H, Hk, dk, dv, slots_n, head_decay;
    float scale;
    long long qs, ks, vs, gs;
    const void *q, *k, *v;
    const float* g;
    float* state;
    const int* slots;
    void* y;
    unsigned* status;
};

template <typename T, int ROWS>  // ROWS: state rows per thread, dk / 8 rounded up
__global__ void __launch_bounds__(128) step_kernel(StepParams p) {
    __shared__ float sq[kMaxDk], sk[kMaxDk];
    __shared__ float4 red[4][16];
    const int b = blockIdx.x;
    const int tiles = (p.dv + kTile - 1) / kTile;
    const int h = blockIdx.y / tiles, c0 = (blockIdx.y - h * tiles) * kTile;
    const int hk = h / (p.H / p.Hk);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, c = c0 + tx * 4;
    const bool in = c < p.dv;
    int slot = p.slots ? p.slots[b] : b;
    const bool bad = slot >= p.slots_n;
    const bool live = slot >= 0 && !bad;
    float4 s[ROWS];
    float* st = live ? p.state + ((size_t)slot * p.H + h) * p.dk * p.dv + c : nullptr;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = ty + 8 * i;
        s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live && in && r < p.dk) s[i] = __ldcs(reinterpret_cast<const float4*>(st + (size_t)r * p.dv));
    }
    // a slot that an earlier row of this call has already is an error: its rows would race
    int again = 0;
    if (p.slots && live)
        for (int i = threadIdx.x; i < b; i += 128) again |= p.slots[i] == slot;
    if (live) {
        for (int i = threadIdx.x; i < p.dk; i += 128) {
            sq[i] = to_f32<T>(((const T*)p.q)[b * p.qs + hk * p.dk + i]);
            sk[i] = to_f32<T>(((const T*)p.k)[b * p.ks + hk * p.dk + i]);
        }
    }
    again = __syncthreads_or(again);
    if ((again || bad) && p.status && threadIdx.x == 0) set_status(p.status, kStatusIndex);
    const bool use = live && !again;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (use && in) {
        float v[4];
        load_vec<T, 4, false>((const T*)p.v + b * p.vs + (long long)h * p.dv + c, v);
        const float a = expf(p.head_decay ? p.g[h] : p.g[b * p.gs + h]);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int r = ty + 8 * i;
            if (r < p.dk) {
                const float k = sk[r], q = sq[r];
                s[i] = make_float4(fmaf(a, s[i].x, k * v[0]), fmaf(a, s[i].y, k * v[1]), fmaf(a, s[i].z, k * v[2]),
                                   fmaf(a, s[i].w, k * v[3]));
                acc.x = fmaf(q, s[i].x, acc.x);
                acc.y = fmaf(q, s[i].y, acc.y);
                acc.z = fmaf(q, s[i].z, acc.z);
                acc.w = fmaf(q, s[i].w, acc.w);
                __stcs(reinterpret_cast<float4*>(st + (size_t)r * p.dv), s[i]);
            }
        }
    }
    // the eight row groups: two in each warp, four warps
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
    if ((threadIdx.x & 16) == 0) red[threadIdx.x >> 5][tx] = acc;
    __syncthreads();
    if (threadIdx.x < 16 && in) {
        float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 r = red[i][tx];
            o[0] += r.x; o[1] += r.y; o[2] += r.z; o[3] += r.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] *= p.scale;
        store_vec<T, 4>((T*)p.y + ((size_t)b * p.H + h) * p.dv + c, o);
    }
}

// ---- host ------------------------------------------------------------------------------------------
size_t type_size(int t) { return t == FV_TYPE_F32 ? 4 : 2; }
long long round_to(long long v, long long m) { return (v + m - 1) / m * m; }

fv_status check_sizes(int N, long long T, int H, int Hk, int dk, int dv, int type, unsigned flags, float scale) {
    if (N < 0 || T < 0 || H < 1 || Hk < 1 || H % Hk != 0) return FV_ERR_SHAPE;
    if (dk < 8 || dk % 8 != 0 || dv < 8 || dv % 8 != 0) return FV_ERR_SHAPE;
    if (type != FV_TYPE_F32 && type != FV_TYPE_BF16) return FV_ERR_SHAPE;
    if (flags & ~(unsigned)FV_LA_HEAD_DECAY) return FV_ERR_SHAPE;
    if (!(scale >= -3.0e38f && scale <= 3.0e38f)) return FV_ERR_SHAPE;
    if (dk > kMaxDk || dv > kMaxDv || H > 4096) return FV_ERR_UNSUPPORTED;
    return FV_OK;
}
// A token stride: 0 = contiguous, else at least a token and a multiple of 16 bytes.
bool stride_ok(long long s, long long width, size_t size) {
    return s == 0 || (s >= width && s * (long long)size % 16 == 0 && s < (1ll << 38));
}

struct Call {
    Shape sh;
    long long rows;  // rows of q, k, v, y
};

fv_status make_call(const fv_linattn_args* a, Call* c) {
    if (!a) return FV_ERR_NULL;
    fv_status s = check_sizes(a->N, a->T, a->H, a->Hk, a->dk, a->dv, a->type, a->flags, a->scale);
    if (s != FV_OK) return s;
    Shape& sh = c->sh;
    memset(&sh, 0, sizeof sh);
    sh.N = a->N; sh.T = a->T; sh.H = a->H; sh.Hk = a->Hk; sh.dk = a->dk; sh.dv = a->dv;
    sh.packed = a->cu_seqlens != nullptr;
    sh.head_decay = (a->flags & FV_LA_HEAD_DECAY) != 0;
    sh.scale = a->scale;
    const size_t e = type_size(a->type);
    const long long wq = (long long)a->Hk * a->dk, wv = (long long)a->H * a->dv;
    if (!stride_ok(a->q_stride, wq, e) || !stride_ok(a->k_stride, wq, e) || !stride_ok(a->v_stride, wv, e) ||
        !stride_ok(a->dy_stride, wv, e))
        return FV_ERR_SHAPE;
    if (a->g_stride != 0 && (a->g_stride < a->H || sh.head_decay || a->g_stride >= (1ll << 40))) return FV_ERR_SHAPE;
    sh.qs = a->q_stride ? a->q_stride : wq;
    sh.ks = a->k_stride ? a->k_stride : wq;
    sh.vs = a->v_stride ? a->v_stride : wv;
    sh.ys = a->dy_stride ? a->dy_stride : wv;
    sh.gs = a->g_stride ? a->g_stride : a->H;
    c->rows = sh.packed ? a->T : (long long)a->N * a->T;
    if (c->rows >= (1ll << 31) || (long long)a->N * a->H >= (1ll << 31)) return FV_ERR_UNSUPPORTED;
    return FV_OK;
}

size_t span(long long rows, long long stride, long long width, size_t size) {
    return rows > 0 ? ((size_t)(rows - 1) * stride + width) * size : 0;
}

fv_status check_tensors(const fv_linattn_args* a, const Call& c, bool grad) {
    const Shape& sh = c.sh;
    if (c.rows > 0 && (!a->q || !a->k || !a->v || !a->g)) return FV_ERR_NULL;
    const void* ps[] = {a->q, a->k, a->v, a->initial_state, a->y, a->final_state};
    for (const void* p : ps)
        if (!ptr_aligned16(p)) return FV_ERR_ALIGN;
    if (((uintptr_t)a->g & 3u) || ((uintptr_t)a->cu_seqlens & 3u)) return FV_ERR_ALIGN;
    if (grad) return FV_OK;
    if (c.rows > 0 && !a->y) return FV_ERR_NULL;
    const size_t e = type_size(a->type);
    const long long wq = (long long)sh.Hk * sh.dk, wv = (long long)sh.H * sh.dv;
    const size_t ny = (size_t)c.rows * wv * e, nst = (size_t)sh.N * sh.H * sh.dk * sh.dv * 4;
    const size_t ng = sh.head_decay ? (size_t)sh.H * 4 : span(c.rows, sh.gs, sh.H, 4);
    const void* in[] = {a->q, a->k, a->v, a->g, a->cu_seqlens, a->initial_state};
    const size_t ni[] = {span(c.rows, sh.qs, wq, e), span(c.rows, sh.ks, wq, e), span(c.rows, sh.vs, wv, e), ng,
                         ((size_t)sh.N + 1) * 4, nst};
    for (int i = 0; i < 6; ++i) {
        if (ranges_overlap(a->y, ny, in[i], ni[i])) return FV_ERR_ALIAS;
        // the final states may replace the initial ones: each element is read before it is written
        if (ranges_overlap(a->final_state, nst, in[i], ni[i]) && !(i == 5 && a->final_state == a->initial_state))
            return FV_ERR_ALIAS;
    }
    if (ranges_overlap(a->y, ny, a->final_state, nst)) return FV_ERR_ALIAS;
    return FV_OK;
}

// Pieces of L tokens (a multiple of the chunk).
fv_status set_pieces(Call* c, long long L) {
    Shape& sh = c->sh;
    sh.L = (int)L;
    sh.per_seq = sh.packed ? 0 : sh.T > 0 ? (int)((sh.T + L - 1) / L) : 1;
    const long long pieces = sh.packed ? sh.T / L + sh.N : (long long)sh.N * sh.per_seq;
    // blocks of the forward, one-dimensional
    if (pieces * sh.H * ((sh.dv + kTile - 1) / kTile) >= (1ll << 31)) return FV_ERR_UNSUPPORTED;
    sh.pieces = (int)pieces;
    return FV_OK;
}

// Length of a forward piece.  One block takes a (piece, head, 64 columns).  Whole sequences need one pass
// over k and v; pieces need a second one and a state each.
//   bf16: a block that shares its SM (148) takes 8100 cycles a chunk, one alone 6900, so a sequence is cut into
// as many pieces as all run at the same time, two blocks on an SM: 12 heads of 128 x 128 over 16384 tokens
// take 113 us in 12 pieces (288 blocks), some 150 us in 8 or in 16; over 4096 tokens 49 us in 11, 64 us in 4.  It
// stays whole where that is shorter than walking a piece twice and the time of three chunks that the second
// launch and the states cost: 4 heads over 512 tokens 21 us whole and cut, over 768 tokens 28 us whole, 22 us
// cut; 4 x 768 tokens of 20 heads 30 us whole, 32 us in three pieces; 4 x 4096 tokens of 24 heads 116 us whole,
// 89 us in three.
//   fp32: bound by the arithmetic of its chunks, so single chunks pay as long as SMs are short of blocks: up to
// about two waves of two blocks on each (1024 tokens of 12 heads: 26 us in pieces of 64, 33 us of 128).
//   packed: the host does not know the lengths.  A sequence is cut where it would take longer than its share
// of all SMs; the pieces start in the order of their lengths (40 sequences of 1 to some 5000 tokens, 24 heads:
// 386 us in pieces of 2048 as they come, 321 us by length, 300 us uncut by length).
constexpr int kSms = 148;
long long forward_piece(const Shape& sh, long long rows, bool f32) {
    const long long unit = f32 ? kC : kTcC;
    const long long whole = sh.T > 0 ? round_to(sh.T, unit) : unit;
    const long long tiles = (long long)sh.H * ((sh.dv + kTile - 1) / kTile);
    if (f32) {
        if (!sh.packed && sh.N * tiles >= kSms) return whole;
        const long long L = round_to((rows * tiles + 4 * kSms - 1) / (4 * kSms), unit);
        return L < unit ? unit : L < whole ? L : whole;
    }
    long long L = whole;
    if (!sh.packed || sh.N == 1) {
        const long long at_once = sh.N > 0 ? 2 * kSms / (sh.N * tiles) : 0;
        if (at_once > 1) L = round_to((sh.T + at_once - 1) / at_once, unit);
    } else {
        L = round_to((rows * tiles + kSms - 1) / kSms, unit);
        if (L < 2 * unit) L = 2 * unit;
    }
    return 2 * L + 3 * unit <= whole ? L : whole;
}

struct Region {
    size_t off;
    size_t take(size_t bytes) {
        const size_t at = off;
        off = round_up256(off + bytes);
        return at;
    }
};
struct Layout {
    size_t control, first_of, table, order, cut, states, dstates, decay, pq, pk, dg, total;
};

bool split(const Call& c) { return c.sh.packed ? c.sh.L < c.sh.T : c.sh.per_seq > 1; }

Layout layout_of(const Call& c, bool grad) {
    const Shape& sh = c.sh;
    Layout l;
    memset(&l, 0, sizeof l);
    Region r{0};
    l.control = r.take(256);
    if (sh.packed) {
        l.first_of = r.take(((size_t)sh.N + 1) * 4);
        l.table = r.take((size_t)sh.pieces * sizeof(Piece));
        if (!grad) l.order = r.take((size_t)sh.pieces * 4);
        if (!grad && split(c)) l.cut = r.take((size_t)sh.pieces * 4);
    }
    const size_t st = (size_t)sh.pieces * sh.H * sh.dk * sh.dv * 4;
    if (grad || split(c)) {
        l.states = r.take(st);
        l.decay = r.take((size_t)sh.pieces * sh.H * 4);
    }
    if (grad) {
        l.dstates = r.take(st);
        if (sh.Hk != sh.H) {
            l.pq = r.take((size_t)c.rows * sh.H * sh.dk * 4);
            l.pk = r.take((size_t)c.rows * sh.H * sh.dk * 4);
        }
        if (sh.head_decay) l.dg = r.take((size_t)sh.pieces * sh.H * 4);
    }
    l.total = r.off;
    return l;
}

fv_status plan_forward(const fv_linattn_args* a, Call* c) {
    fv_status s = make_call(a, c);
    if (s != FV_OK) return s;
    if ((s = set_pieces(c, forward_piece(c->sh, c->rows, a->type == FV_TYPE_F32))) != FV_OK) return s;
    // Up to four pieces add up the states before them by themselves: a few reads from L2 in place of a launch that
    // reads and writes every state.  bf16, 4 pieces: 64 us against 75 us (12 heads of 128 x 128), 36 us against 38
    // us (16 of 64 x 64); 8 pieces 32 us against 31 us, 16 pieces 63 us against 29 us.  fp32, 4 pieces: alike on
    // the card, a launch less (3 us) for the host; 16 pieces 33 us against 26 us.  Not where the final states
    // replace the initial ones, which every piece then reads while the last one writes.
    c->sh.look_back = !c->sh.packed && c->sh.per_seq > 1 && c->sh.per_seq <= 4 &&
                      !(a->final_state && a->final_state == a->initial_state);
    return FV_OK;
}
fv_status plan_grad(const fv_linattn_args* a, Call* c) {
    fv_status s = make_call(a, c);
    if (s != FV_OK) return s;
    return set_pieces(c, a->type == FV_TYPE_F32 ? kC : kTcC);  // the kernels' chunks
}

bool good_ws(const void* ws, size_t bytes, size_t need) { return ws && ((uintptr_t)ws & 255u) == 0 && bytes >= need; }

fv_status start_call(const fv_linattn_args* a, const Call& c, const Layout& l, char* ws, PackedPlan* plan, cudaStream_t st) {
    int* control = (int*)(ws + l.control);
    memset(plan, 0, sizeof *plan);
    if (!c.sh.packed) {
        if (a->type == FV_TYPE_F32 && c.sh.N > 0) return FV_OK;  // no wait to give up: the first kernel clears it
        const cudaError_t e = cudaMemsetAsync(control, 0, 4, st);
        if (e == cudaSuccess) return FV_OK;
        note_cuda_error(e, "status reset");
        return FV_ERR_CUDA;
    }
    plan->count = control + 1;
    plan->first_of = (const int*)(ws + l.first_of);
    plan->table = (const Piece*)(ws + l.table);
    plan->order = l.order ? (const int*)(ws + l.order) : nullptr;
    plan_kernel<<<1, 1024, 0, st>>>(a->cu_seqlens, c.sh.N, c.sh.T, c.sh.L, c.sh.pieces, control, (int*)(ws + l.first_of),
                                    (Piece*)(ws + l.table), (int*)plan->order, l.cut ? (int*)(ws + l.cut) : nullptr);
    return launch_status("plan_kernel");
}

// The driver's tensor-map encoder, asked from the runtime once (the library does not link the driver).
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encoder() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
        return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? (EncodeTiled)p : nullptr;
    }();
    return fn;
}
// bf16 [rows][heads][d] with `stride` elements between rows, in boxes of 128 rows of 64 channels of one
// head, 128-byte swizzle.  Base and strides are multiples of 16 bytes (checked), as is each box's start
// (d is a multiple of 8).
fv_status make_map(CUtensorMap* m, const void* p, long long rows, int heads, int d, long long stride) {
    const EncodeTiled fn = encoder();
    if (!fn) {
        note_cuda_error(cudaErrorNotSupported, "cuTensorMapEncodeTiled");
        return FV_ERR_CUDA;
    }
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, kTcC}, one[3] = {1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, one,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return FV_OK;
    note_cuda_error(cudaErrorInvalidValue, "cuTensorMapEncodeTiled");
    return FV_ERR_CUDA;
}

fv_status make_maps(TcMaps* maps, const Call& c, const Tensors& x, const void* y, long long y_stride) {
    memset(maps, 0, sizeof *maps);
    fv_status s = FV_OK;
    if (c.rows == 0 || (s = make_map(&maps->q, x.q, c.rows, c.sh.Hk, c.sh.dk, c.sh.qs)) != FV_OK ||
        (s = make_map(&maps->k, x.k, c.rows, c.sh.Hk, c.sh.dk, c.sh.ks)) != FV_OK ||
        (s = make_map(&maps->v, x.v, c.rows, c.sh.H, c.sh.dv, c.sh.vs)) != FV_OK || !y)
        return s;
    return make_map(&maps->y, y, c.rows, c.sh.H, c.sh.dv, y_stride);
}

// Launches a kernel; `overlap`: it may begin once every block of the launch before it has let it or has ended,
// and waits in the kernel for that launch's results.
template <typename... P, typename... A>
fv_status launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, bool overlap, const char* where,
                       const A&... args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = overlap ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e == cudaSuccess) return launch_status(where);
    note_cuda_error(e, where);
    return FV_ERR_CUDA;
}

// fp32 runs on FMAs, bf16 on the tensor cores; one block per (piece, head, 64 columns of v) in both.
template <typename T, int DK, bool OUT>
fv_status launch_pass(const Call& c, const PackedPlan& pl, const Tensors& x, const float* start, float* loc, float* decay,
                      unsigned* status, cudaStream_t st) {
    // a sequence that is cut has more than L tokens, so at most twice its share of T / L pieces
    const int pieces = !OUT && c.sh.packed ? (int)std::min<long long>(c.sh.pieces, 2ll * c.sh.T / c.sh.L) : c.sh.pieces;
    const unsigned grid = (unsigned)pieces * c.sh.H * ((c.sh.dv + kTile - 1) / kTile);
    // the outputs' blocks begin while the states' (and the joining pass's) still run, and wait for them before
    // they read one
    const bool overlap = OUT && split(c);
    if constexpr (sizeof(T) == 4) {
        constexpr size_t smem = fwd_smem<DK>();
        const fv_status s = opt_in_smem<simt_kernel<DK, OUT>>(smem, "linattn forward");
        if (s != FV_OK) return s;
        return launch_after(simt_kernel<DK, OUT>, dim3(grid), kThr, smem, st, overlap, "linattn forward", c.sh, pl, x, start, loc,
                            decay, status);
    } else {
        TcMaps maps;
        const fv_status m = make_maps(&maps, c, x, OUT ? x.y : nullptr, (long long)c.sh.H * c.sh.dv);
        if (m != FV_OK) return m;
        constexpr size_t smem = TcSmem<DK>::bytes;
        const fv_status s = opt_in_smem<tc_forward_kernel<DK, OUT>>(smem, "linattn forward");
        if (s != FV_OK) return s;
        return launch_after(tc_forward_kernel<DK, OUT>, dim3(grid), kTcThr, smem, st, overlap, "linattn forward", maps, c.sh, pl, x,
                            start, loc, decay, status);
    }
}
template <typename T, bool OUT>
fv_status forward_pass(const Call& c, const PackedPlan& pl, const Tensors& x, const float* start, float* loc, float* decay,
                       unsigned* status, cudaStream_t st) {
    return c.sh.dk <= 64 ? launch_pass<T, 64, OUT>(c, pl, x, start, loc, decay, status, st)
                         : launch_pass<T, 128, OUT>(c, pl, x, start, loc, decay, status, st);
}

template <typename T>
fv_status forward_t(const Call& c, const Layout& l, const PackedPlan& pl, const Tensors& x, char* ws, cudaStream_t st) {
    unsigned* status = (unsigned*)(ws + l.control);
    if (!split(c)) return forward_pass<T, true>(c, pl, x, nullptr, nullptr, nullptr, status, st);
    float* states = (float*)(ws + l.states);
    float* decay = (float*)(ws + l.decay);
    PackedPlan cut = pl;
    if (c.sh.packed) {
        cut.count = (const int*)(ws + l.control) + 4;
        cut.order = (const int*)(ws + l.cut);
    }
    fv_status s = forward_pass<T, false>(c, cut, x, nullptr, states, decay, status, st);
    if (s != FV_OK) return s;
    if (!c.sh.look_back) {
        s = launch_after(join_kernel, dim3(c.sh.N * c.sh.H, (c.sh.dk * c.sh.dv / 4 + 255) / 256), 256, 0, st, true, "join_kernel", c.sh,
                         pl.first_of, (const int*)ws, states, (const float*)decay, x.s0, x.st);
        if (s != FV_OK) return s;
    }
    return forward_pass<T, true>(c, pl, x, states, nullptr, decay, status, st);
}

// (1) the chunks' own states, (2) the states entering and the gradients leaving them, (3) the gradients.
template <typename T, int DK>
fv_status grad_dk(const Call& c, const Layout& l, const PackedPlan& pl, const Tensors& x, const GradOut& o, float* ds0, char* ws,
                  cudaStream_t st) {
    float* S = (float*)(ws + l.states);
    float* dS = (float*)(ws + l.dstates);
    float* decay = (float*)(ws + l.decay);
    unsigned* status = (unsigned*)(ws + l.control);
    const int tiles = (c.sh.dv + kTile - 1) / kTile;
    fv_status s;
    [[maybe_unused]] TcMaps maps;
    if constexpr (sizeof(T) == 4) {
        constexpr size_t s1 = local_smem<DK>();
        if ((s = opt_in_smem<simt_local_states_kernel<DK>>(s1, "linattn local states")) != FV_OK) return s;
        simt_local_states_kernel<DK><<<dim3(c.sh.pieces, c.sh.H * tiles, 2), kThr, s1, st>>>(c.sh, pl, x, S, dS, decay, status);
    } else {
        constexpr size_t s1 = TcLocalSmem<DK>::bytes;
        if ((s = make_maps(&maps, c, x, x.dy, c.sh.ys)) != FV_OK) return s;
        if ((s = opt_in_smem<tc_local_kernel<DK>>(s1, "linattn local states")) != FV_OK) return s;
        tc_local_kernel<DK><<<dim3(c.sh.pieces, c.sh.H * tiles, 2), kTcThr, s1, st>>>(maps, c.sh, pl, x, S, dS, decay, status);
    }
    if ((s = launch_status("linattn local states")) != FV_OK) return s;
    // each launch begins while the one before it ends, and waits for it before it reads a state
    s = launch_after(join_grad_kernel, dim3(c.sh.N * c.sh.H, (c.sh.dk * c.sh.dv / 4 + 255) / 256, 2), 256, 0, st, true, "join_grad_kernel",
                     c.sh, pl.first_of, (const int*)ws, S, dS, (const float*)decay, x.s0, x.ds, ds0);
    if (s != FV_OK) return s;
    if constexpr (sizeof(T) == 4) {
        constexpr size_t s2 = grad_smem<DK>();
        if ((s = opt_in_smem<simt_grad_kernel<DK>>(s2, "linattn gradient")) != FV_OK) return s;
        return launch_after(simt_grad_kernel<DK>, dim3(c.sh.pieces, c.sh.H), kThr, s2, st, true, "linattn gradient", c.sh, pl, x,
                            (const float*)S, (const float*)dS, o);
    } else {
        constexpr size_t s2 = TcGradSmem<DK>::bytes;
        if ((s = opt_in_smem<tc_grad_kernel<DK>>(s2, "linattn gradient")) != FV_OK) return s;
        return launch_after(tc_grad_kernel<DK>, dim3(c.sh.pieces, c.sh.H), kTcThr, s2, st, true, "linattn gradient", maps, c.sh, pl, x,
                            (const float*)S, (const float*)dS, o, status);
    }
}

template <typename T>
fv_status grad_t(const Call& c, const Layout& l, const PackedPlan& pl, const Tensors& x, const fv_linattn_grads* g, char* ws,
                 cudaStream_t st) {
    GradOut o;
    o.partial = c.sh.Hk != c.sh.H;
    o.dq = o.partial ? (void*)(ws + l.pq) : g->dq;
    o.dk = o.partial ? (void*)(ws + l.pk) : g->dk;
    o.dv = g->dv;
    o.dg = c.sh.head_decay ? (float*)(ws + l.dg) : g->dg;
    fv_status s = c.sh.dk <= 64 ? grad_dk<T, 64>(c, l, pl, x, o, g->d_initial_state, ws, st)
                                : grad_dk<T, 128>(c, l, pl, x, o, g->d_initial_state, ws, st);
    if (s != FV_OK) return s;
    if (o.partial && c.rows > 0) {
        const long long n = c.rows * c.sh.Hk * c.sh.dk / 4;
        const unsigned blocks = (unsigned)(n / 256 + 1 < 148 * 16 ? n / 256 + 1 : 148 * 16);
        fold_heads_kernel<T><<<dim3(blocks, 2), 256, 0, st>>>(c.sh, (const int*)ws, (const float*)o.dq, (const float*)o.dk,
                                                              (T*)g->dq, (T*)g->dk, c.rows);
        if ((s = launch_status("fold_heads_kernel")) != FV_OK) return s;
    }
    if (c.sh.head_decay) {
        fold_decay_kernel<<<c.sh.H, 256, 0, st>>>(c.sh, (const int*)ws, o.dg, g->dg);
        if ((s = launch_status("fold_decay_kernel")) != FV_OK) return s;
    }
    return FV_OK;
}

fv_status check_grads(const fv_linattn_args* a, const Call& c, const fv_linattn_grads* g) {
    if (!g) return FV_ERR_NULL;
    const Shape& sh = c.sh;
    if (c.rows > 0 && (!g->dy || !g->dq || !g->dk || !g->dv || !g->dg)) return FV_ERR_NULL;
    if (sh.head_decay && !g->dg) return FV_ERR_NULL;
    const void* ps[] = {g->dy, g->dq, g->dk, g->dv, g->d_final_state, g->d_initial_state};
    for (const void* p : ps)
        if (!ptr_aligned16(p)) return FV_ERR_ALIGN;
    if ((uintptr_t)g->dg & 3u) return FV_ERR_ALIGN;
    const size_t e = type_size(a->type);
    const long long wq = (long long)sh.Hk * sh.dk, wv = (long long)sh.H * sh.dv;
    const size_t nq = (size_t)c.rows * wq * e, nv = (size_t)c.rows * wv * e, nst = (size_t)sh.N * sh.H * sh.dk * sh.dv * 4;
    const size_t ng = sh.head_decay ? (size_t)sh.H * 4 : (size_t)c.rows * sh.H * 4;
    const void* out[] = {g->dq, g->dk, g->dv, g->dg, g->d_initial_state};
    const size_t no[] = {nq, nq, nv, ng, nst};
    const void* in[] = {a->q, a->k, a->v, a->g, a->cu_seqlens, a->initial_state, g->dy, g->d_final_state};
    const size_t ni[] = {span(c.rows, sh.qs, wq, e), span(c.rows, sh.ks, wq, e), span(c.rows, sh.vs, wv, e),
                         sh.head_decay ? (size_t)sh.H * 4 : span(c.rows, sh.gs, sh.H, 4), ((size_t)sh.N + 1) * 4, nst,
                         span(c.rows, sh.ys, wv, e), nst};
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < 8; ++j)
            if (ranges_overlap(out[i], no[i], in[j], ni[j]) && !(i == 4 && j == 7 && g->d_initial_state == g->d_final_state))
                return FV_ERR_ALIAS;
        for (int j = i + 1; j < 5; ++j)
            if (ranges_overlap(out[i], no[i], out[j], no[j])) return FV_ERR_ALIAS;
    }
    return FV_OK;
}

template <typename T>
fv_status step_t(const StepParams& p, cudaStream_t st) {
    const dim3 grid(p.B, p.H * ((p.dv + kTile - 1) / kTile));
    if (p.dk <= 32) step_kernel<T, 4><<<grid, 128, 0, st>>>(p);
    else if (p.dk <= 64) step_kernel<T, 8><<<grid, 128, 0, st>>>(p);
    else step_kernel<T, 16><<<grid, 128, 0, st>>>(p);
    return launch_status("linattn step");
}

}  // namespace
}  // namespace la
}  // namespace fv

using namespace fv;

extern "C" {

fv_status fastvim_linattn_validate(const fv_linattn_args* args) {
    la::Call c;
    fv_status s = la::plan_forward(args, &c);
    return s != FV_OK ? s : la::check_tensors(args, c, false);
}

size_t fastvim_linattn_workspace_size(const fv_linattn_args* args) {
    la::Call c;
    return la::plan_forward(args, &c) == FV_OK ? la::layout_of(c, false).total : 0;
}

fv_status fastvim_linattn_forward(const fv_linattn_args* args, void* ws, size_t ws_bytes, void* stream) {
    la::Call c;
    fv_status s = la::plan_forward(args, &c);
    if (s != FV_OK || (s = la::check_tensors(args, c, false)) != FV_OK) return s;
    const la::Layout l = la::layout_of(c, false);
    if (!la::good_ws(ws, ws_bytes, l.total)) return FV_ERR_WORKSPACE;
    cudaStream_t st = (cudaStream_t)stream;
    la::PackedPlan pl;
    if ((s = la::start_call(args, c, l, (char*)ws, &pl, st)) != FV_OK || c.sh.N == 0) return s;
    la::Tensors x{args->q, args->k, args->v, nullptr, args->g, args->initial_state, nullptr, args->y, args->final_state};
    return args->type == FV_TYPE_F32 ? la::forward_t<float>(c, l, pl, x, (char*)ws, st)
                                     : la::forward_t<__nv_bfloat16>(c, l, pl, x, (char*)ws, st);
}

size_t fastvim_linattn_backward_workspace_size(const fv_linattn_args* args) {
    la::Call c;
    return la::plan_grad(args, &c) == FV_OK ? la::layout_of(c, true).total : 0;
}

fv_status fastvim_linattn_backward(const fv_linattn_args* args, const fv_linattn_grads* grads, void* ws, size_t ws_bytes,
                                   void* stream) {
    la::Call c;
    fv_status s = la::plan_grad(args, &c);
    if (s != FV_OK || (s = la::check_tensors(args, c, true)) != FV_OK || (s = la::check_grads(args, c, grads)) != FV_OK) return s;
    const la::Layout l = la::layout_of(c, true);
    if (!la::good_ws(ws, ws_bytes, l.total)) return FV_ERR_WORKSPACE;
    cudaStream_t st = (cudaStream_t)stream;
    la::PackedPlan pl;
    if ((s = la::start_call(args, c, l, (char*)ws, &pl, st)) != FV_OK) return s;
    if (c.sh.N == 0) {
        if (!c.sh.head_decay) return FV_OK;
        const cudaError_t e = cudaMemsetAsync(grads->dg, 0, (size_t)c.sh.H * 4, st);
        if (e == cudaSuccess) return FV_OK;
        note_cuda_error(e, "gradient reset");
        return FV_ERR_CUDA;
    }
    la::Tensors x{args->q, args->k, args->v, grads->dy, args->g, args->initial_state, grads->d_final_state, nullptr, nullptr};
    return args->type == FV_TYPE_F32 ? la::grad_t<float>(c, l, pl, x, grads, (char*)ws, st)
                                     : la::grad_t<__nv_bfloat16>(c, l, pl, x, grads, (char*)ws, st);
}

fv_status fastvim_linattn_step(const fv_linattn_step_args* args, void* stream) {
    if (!args) return FV_ERR_NULL;
    const fv_linattn_step_args& a = *args;
    fv_status s = la::check_sizes(a.B, 1, a.H, a.Hk, a.dk, a.dv, a.type, a.flags, a.scale);
    if (s != FV_OK) return s;
    const size_t e = la::type_size(a.type);
    const long long wq = (long long)a.Hk * a.dk, wv = (long long)a.H * a.dv;
    if (!la::stride_ok(a.q_stride, wq, e) || !la::stride_ok(a.k_stride, wq, e) || !la::stride_ok(a.v_stride, wv, e)) return FV_ERR_SHAPE;
    const bool head = (a.flags & FV_LA_HEAD_DECAY) != 0;
    if (a.g_stride != 0 && (a.g_stride < a.H || head || a.g_stride >= (1ll << 40))) return FV_ERR_SHAPE;
    if (a.S < 0 || (!a.slots && a.S < a.B)) return FV_ERR_SHAPE;
    if (a.B == 0) return FV_OK;
    if (!a.q || !a.k || !a.v || !a.g || !a.y || (a.S > 0 && !a.state)) return FV_ERR_NULL;
    const void* ps[] = {a.q, a.k, a.v, a.state, a.y};
    for (const void* p : ps)
        if (!ptr_aligned16(p)) return FV_ERR_ALIGN;
    if (((uintptr_t)a.g & 3u) || ((uintptr_t)a.slots & 3u) || ((uintptr_t)a.status & 3u)) return FV_ERR_ALIGN;
    la::StepParams p;
    memset(&p, 0, sizeof p);
    p.B = a.B; p.H = a.H; p.Hk = a.Hk; p.dk = a.dk; p.dv = a.dv; p.slots_n = a.S; p.head_decay = head;
    p.scale = a.scale;
    p.qs = a.q_stride ? a.q_stride : wq;
    p.ks = a.k_stride ? a.k_stride : wq;
    p.vs = a.v_stride ? a.v_stride : wv;
    p.gs = a.g_stride ? a.g_stride : a.H;
    p.q = a.q; p.k = a.k; p.v = a.v; p.g = a.g; p.state = a.state; p.slots = a.slots; p.y = a.y; p.status = a.status;
    const size_t ny = (size_t)a.B * wv * e, nst = (size_t)a.S * a.H * a.dk * a.dv * 4;
    const void* in[] = {a.q, a.k, a.v, a.g, a.slots, a.status};
    const size_t ni[] = {la::span(a.B, p.qs, wq, e), la::span(a.B, p.ks, wq, e), la::span(a.B, p.vs, wv, e),
                         head ? (size_t)a.H * 4 : la::span(a.B, p.gs, a.H, 4), (size_t)a.B * 4, 4};
    for (int i = 0; i < 6; ++i)
        if (ranges_overlap(a.y, ny, in[i], ni[i]) || ranges_overlap(a.state, nst, in[i], ni[i])) return FV_ERR_ALIAS;
    if (ranges_overlap(a.y, ny, a.state, nst)) return FV_ERR_ALIAS;
    return a.type == FV_TYPE_F32 ? la::step_t<float>(p, (cudaStream_t)stream) : la::step_t<__nv_bfloat16>(p, (cudaStream_t)stream);
}

}  // extern "C"
