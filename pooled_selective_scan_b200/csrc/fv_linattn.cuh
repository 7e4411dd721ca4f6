// fv_linattn.cuh -- shared definitions of the linear-attention kernels (sm_100a).
//
// Per sequence and value head h, with the key head h Hk / H of its group:
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T      (dk x dv, fp32),       y_t = scale S_t^T q_t.
// A chunk of C tokens with G_i = sum_{t <= i} g_t taken inside the chunk is
//   y_i   = scale (e^{G_i} S_in^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j)
//   S_out = e^{G_C} S_in + sum_j e^{G_C - G_j} k_j v_j^T,
// products of matrices whose weights are all at most 1 when g <= 0: no factor e^{-G_j} appears.
#pragma once

#include "fv_common.cuh"
#include "fv_types.cuh"

namespace fv {
namespace la {

constexpr int kTile = 64;     // columns of v per block
constexpr int kMaxDk = 128;
constexpr int kMaxDv = 256;

// A run of consecutive tokens of one sequence; its place in the state buffers is its number among all pieces.
struct Piece {
    int seq, row, len, flags;  // row: first token's row; flags: 1 first, 2 last piece of its sequence
};

struct Shape {
    int N, T, H, Hk, dk, dv;
    int packed, head_decay;  // cu_seqlens given; g is [H]
    float scale;
    long long qs, ks, vs, gs, ys;  // elements between tokens (ys: dy)
    int L;                         // tokens per piece
    int per_seq;                   // pieces per sequence (dense)
    int pieces;                    // pieces in all (packed: at most)
    int look_back;                 // pieces add up the states before them by themselves (no joining pass)
};

struct Tensors {
    const void *q, *k, *v, *dy;
    const float* g;
    const float *s0, *ds;
    void* y;
    float* st;
};

struct PackedPlan {
    const int* count;     // pieces to do
    const Piece* table;   // [pieces]
    const int* first_of;  // [N + 1] first piece of each sequence
    const int* order;     // the pieces to do: all, long ones first, or those of sequences that are cut; null: as they are
};

// The i-th piece, and its number `id` (its place in the state buffers).
__device__ __forceinline__ bool get_piece(const Shape& sh, const PackedPlan& pl, int i, Piece& p, int& id) {
    id = i;
    if (sh.packed) {
        if (i >= *pl.count) return false;
        if (pl.order) id = pl.order[i];
        p = pl.table[id];
        return true;
    }
    const int n = i / sh.per_seq, c = i - n * sh.per_seq;
    const int t0 = c * sh.L;
    p.seq = n;
    p.row = n * sh.T + t0;
    p.len = min(sh.L, sh.T - t0);
    p.flags = (c == 0 ? 1 : 0) | (c == sh.per_seq - 1 ? 2 : 0);
    return true;
}

// Sums of log decays as base-2 exponents in two parts, hi a whole number and lo in [0, 1): a difference
// (hi_i - hi_j) + (lo_i - lo_j) is then as exact for tokens behind a strong decay as for the first ones,
// where one fp32 sum would lose the small steps.
struct Exponent {
    float hi, lo;
};
__device__ __forceinline__ float decay_between(const Exponent& i, const Exponent& j) {
    return ex2_approx((i.hi - j.hi) + (i.lo - j.lo));
}
// The power of a sum by its two parts: of hi + lo in one number, what its last bit leaves (2^-18 at 64 to 128) would be
// the power's error, however small the other sums are that it is multiplied with.
__device__ __forceinline__ float power_of(float hi, float lo) {
    return ex2_approx(lo) * __int_as_float(((int)fminf(fmaxf(hi, -127.f), 127.f) + 127) << 23);
}
// The decay of a whole run of tokens, which a state takes over and over: the approximate power is off by up to
// 2^-22, always to the same side where the decays are all alike, and a state of a long memory adds that up.
// e^x by its series to x^7, |x| <= ln 2 / 2: the rest is below 6e-9 of it.
__device__ __forceinline__ float decay_of(const Exponent& e) {
    const float n = rintf(e.lo), x = ((e.lo - n) * 0.693147181f), k = e.hi + n;
    float p = 1.f / 5040.f;
    p = fmaf(p, x, 1.f / 720.f);
    p = fmaf(p, x, 1.f / 120.f);
    p = fmaf(p, x, 1.f / 24.f);
    p = fmaf(p, x, 1.f / 6.f);
    p = fmaf(p, x, 0.5f);
    p = fmaf(p, x, 1.f);
    p = fmaf(p, x, 1.f);
    return p * (k < -126.f ? 0.f : k > 127.f ? __int_as_float(0x7f800000) : __int_as_float(((int)k + 127) << 23));
}
// The square root of a run's decay.  A chunk's e^{G_C} <dS, S> takes one with each factor: the product of two
// large states may leave fp32, and so may the decay, where all three together are of ordinary size.
__device__ __forceinline__ float root_decay_of(const Exponent& e) {
    const float h = floorf(0.5f * e.hi);
    return decay_of(Exponent{h, 0.5f * ((e.hi - 2.f * h) + e.lo)});
}
// For a warp's 32 tokens at once, one a lane, in whole numbers: the exponent g log2 e is split into its
// nearest whole number, a fraction in units of 2^-26 (a sum of 32 fits 32 bits), whose running sums are
// exact, and what the units leave, at most 2^-27 (a decay that is the same for every token leaves the same
// every time: 32 of them would be 2^-22).  A 64-bit floating-point scan took ten times as long.
// NaN anywhere makes `bad`.
struct FixedSum {
    int hi, lo;
    float rest;
};
template <int BITS>
__device__ __forceinline__ FixedSum fixed_exponent(float g) {
    const float v = fminf(fmaxf(g, -200.f), 200.f);  // 2^+-288 is 0 or infinity in fp32
    const float p = v * 1.44269504f;
    const float err = fmaf(v, 1.44269504f, -p) + v * 1.92596299e-8f;  // log2 e to 48 bits
    const float r = rintf(p), f = (p - r) + err, u = rintf(f * (float)(1 << BITS));
    // f and err have their own roundings; the rest of f is taken before they are added up
    return FixedSum{(int)r, (int)u, ((p - r) - u * (1.f / (float)(1 << BITS))) + err};
}
__device__ __forceinline__ void warp_scan(FixedSum& s) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, s.hi, o), b = __shfl_up_sync(0xffffffffu, s.lo, o);
        const float c = __shfl_up_sync(0xffffffffu, s.rest, o);
        if ((int)(threadIdx.x & 31) >= o) {
            s.hi += a;
            s.lo += b;
            s.rest += c;
        }
    }
}
template <int BITS>
__device__ __forceinline__ Exponent exponent_of(int hi, int lo, float rest) {
    const int carry = lo >> BITS;
    return Exponent{(float)(hi + carry), fmaf((float)(lo - (carry << BITS)), 1.f / (float)(1 << BITS), rest)};
}
struct WarpSums {
    Exponent own;    // sum up to this lane's token
    float to_end;    // from behind it to the last token's
    Exponent total;
    bool bad;
};
__device__ __forceinline__ WarpSums warp_sums(float g) {
    FixedSum f = fixed_exponent<26>(g);
    warp_scan(f);
    const int thi = __shfl_sync(0xffffffffu, f.hi, 31), tlo = __shfl_sync(0xffffffffu, f.lo, 31);
    const float trest = __shfl_sync(0xffffffffu, f.rest, 31);
    WarpSums s;
    s.own = exponent_of<26>(f.hi, f.lo, f.rest);
    const Exponent e = exponent_of<26>(thi - f.hi, tlo - f.lo, trest - f.rest);
    s.to_end = e.hi + e.lo;
    s.total = exponent_of<26>(thi, tlo, trest);
    s.bad = __any_sync(0xffffffffu, g != g);
    return s;
}
// A chunk of the tensor-core kernels with a log decay above kRise (32 tokens of it are less than one doubling) takes a
// power for each weight, from these sums, in place of products of quarters' powers (see fv_linattn_tc.cuh).
constexpr float kRise = 0.015625f;
// The sum from the chunk's first token up to this lane's one of `quarter`, and that of all its 128 tokens; g, step and n:
// the chunk's first token, the elements between tokens, and how many there are.  NaN anywhere makes both NaN.  A
// function of its own, as what is used in such a chunk alone is: inline it took registers from all calls (8 x 4096 tokens
// x 12 heads of 64, gradient: 300 us for 283 us).
struct ChunkSum {
    Exponent at, total;
};
__device__ __noinline__ ChunkSum chunk_sum(const float* g, long long step, int n, int quarter) {
    ChunkSum s{{0.f, 0.f}, {0.f, 0.f}};
    bool bad = false;
#pragma unroll 1
    for (int m = 0; m < 4; ++m) {
        const int t = 32 * m + (threadIdx.x & 31);
        const WarpSums w = warp_sums(t < n ? __ldg(g + t * step) : 0.f);
        bad |= w.bad;
        if (m == quarter) s.at = Exponent{s.total.hi + w.own.hi, s.total.lo + w.own.lo};
        s.total.hi += w.total.hi;
        s.total.lo += w.total.lo;
    }
    if (bad) s.at.lo = s.total.lo = __int_as_float(0x7fffffff);
    return s;
}
// The power of the sum from behind `at` up to `total`.
__device__ __forceinline__ float decay_behind(const Exponent& at, const Exponent& total) {
    return decay_of(Exponent{total.hi - at.hi, total.lo - at.lo});
}

// A kernel launched to overlap the one before it: lets the next begin, and waits for the one before to end
// (returns at once in a launch without the overlap).  What the launch before writes is read by loads that see
// other kernels' stores (cp.async, __ldcg, __ldcs) through pointers that promise nothing: __ldg, or a const
// __restrict__ pointer, asks for memory that nobody writes as long as the kernel runs, and may be read ahead of the wait.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" : : : "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" : : : "memory"); }

// Four values at offset `at` of the state entering piece `id` of a sequence, where the joining pass is left
// out: run = initial; for the pieces before: run = decay run + own.
__device__ __forceinline__ float4 look_back(const Shape& sh, const float* own, const float* decay, const float* s0, int id, int seq,
                                            int h, size_t at) {
    const size_t size = (size_t)sh.dk * sh.dv;
    float4 run = s0 ? __ldg(reinterpret_cast<const float4*>(s0 + ((size_t)seq * sh.H + h) * size + at)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = seq * sh.per_seq; p < id; ++p) {
        const float d = __ldcg(decay + (size_t)p * sh.H + h);
        const float4 v = __ldcg(reinterpret_cast<const float4*>(own + ((size_t)p * sh.H + h) * size + at));
        run = make_float4(fmaf(d, run.x, v.x), fmaf(d, run.y, v.y), fmaf(d, run.z, v.z), fmaf(d, run.w, v.w));
    }
    return run;
}

__device__ __forceinline__ int key_head(const Shape& sh, int h) { return h / (sh.H / sh.Hk); }

}  // namespace la
}  // namespace fv
