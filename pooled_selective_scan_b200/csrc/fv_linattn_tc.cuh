// fv_linattn_tc.cuh -- the bf16 forward of linear attention on the 5th-generation tensor cores.
//
// One block walks the chunks (128 tokens) of one piece, head and 64 columns of v, with the state in
// registers.  Per chunk, with T x T scores A = Q K^T, local decays u and w (below) and S = S_in:
//   tensor cores:  A = Q K^T;  O1 = Q S           (S as two bf16 tiles, hi + lo)
//   threads:       V~ = e^{G_C - G_j} v_j         (one or three bf16 parts)
//   tensor cores:  D = K^T V~
//   threads:       P = A * w                      (causal, bf16, into tensor memory)
//   tensor cores:  O2 = P V                       (A operand in tensor memory)
//   threads:       S = e^{G_C} S + D, split into hi + lo tiles again;  y = scale (e^{G_i} O1 + O2).
// Each product runs while the threads work at the step before its result is needed.  Accumulators are
// fp32 in tensor memory (256 columns: A, then O2 over its lower and P over its upper half; O1; D).  What is
// rounded to bf16: the weighted scores, once (they meet bf16 values and a bf16 result; in two parts in a chunk
// of up to 64 tokens), and the weighted v where only y follows: y then has two roundings of at most 2^-8 per
// term, its own included.  A caller
// who reads the fp32 state back gets one that is exact to fp32's order: the state is then a sum of exact
// bf16 k times weighted v in three bf16 parts (two would leave 2.4e-6).  Where the state is an
// operand it goes in as two parts.  Parts cost shared-memory traffic (each is written once and read, with
// k, by the products), which bounds the kernel together with the load latency of a chunk.
//
// Weights: with local sums L_i inside each 32-token quarter (one warp's lanes; T_q its total), pairs of
// quarters q > p weigh exp2(L_i) times the decays of the quarters between times u_j = exp2(T_p - L_j): two
// multiplications by numbers of the row and the column, where an exponential per pair would take the
// special-function units longer than the products take.  Every factor is at most 1.  Pairs in one
// quarter take exp2(L_i - T_q) u_j, the first at most 2^100; a quarter that decays further takes each
// exponential by itself.  So do all pairs of a chunk with a log decay above kRise: there the factors, sums over other
// tokens than the pair's own, could leave fp32 where the pair's weight does not (16 x 4096 tokens x 12 heads of 64,
// every chunk such a one: 321 us for 143 us; gradient of 8: 375 us for 283 us).
//
// Loads are TMA boxes of 128 tokens x 64 channels of one head (one thread issues them; channels behind the
// head's read zero); the rows behind a sequence's last token, which belong to the next, are zeroed in
// shared memory.  The threads' arithmetic is what bounds the kernel: pairs of fp32 values share an
// instruction where they can.
//
// 16 x 4096 tokens x 12 heads of 64 x 64: 142 us, where its traffic would take 62 us and the products 43 us of
// the tensor cores' rate; of the time, the weighted v takes about 15 %, y's way out 17 %, the scores 8 %, all
// products 5 %.  dk <= 64 has its own form: with the one for 128, the same call takes 151 us (gradient of 8 381 us
// for 282 us; fp32, 8 x 1024 tokens x 6 heads of 64 x 64, 99 us for 67 us, gradient 232 us for 148 us).
//
// Layout: 256 threads; warp w reads tensor-memory lanes 32 (w % 4) .. + 31 (its 32 tokens, or state
// rows) and the column half w / 4.  112 KB of tiles: Q, K, V, S and, over Q and S where dk > 64, V~ -- two
// blocks on an SM, so that one's barriers and products overlap the other's arithmetic.
#pragma once

#include "fv_linattn.cuh"
#include "fv_tc.cuh"

namespace fv {
namespace la {

constexpr int kTcC = 128;
constexpr int kTcThr = 256;
constexpr uint32_t kTileBytes = kTcC * 128;  // 128 rows of 64 bf16 values

template <int DK>
struct TcSmem {
    static constexpr uint32_t kBlocks = DK / 64;
    static constexpr uint32_t q = 0;
    static constexpr uint32_t k = kBlocks * kTileBytes;
    static constexpr uint32_t v = 2 * kBlocks * kTileBytes;
    static constexpr uint32_t s = v + kTileBytes + (DK == 64 ? 3 * kTileBytes : 0);  // S: hi, lo
    static constexpr uint32_t slo = s + DK * 128;
    // V~'s parts: behind V, or over Q and S
    static constexpr uint32_t vhi = DK == 64 ? v + kTileBytes : q;
    static constexpr uint32_t vmid = vhi + kTileBytes;
    static constexpr uint32_t vlo = DK == 64 ? vmid + kTileBytes : s;
    static constexpr uint32_t y = DK == 64 ? vmid : v;  // the outputs on their way out
    static constexpr uint32_t u = s + 2 * DK * 128;     // float [128]
    static constexpr uint32_t dec = u + kTcC * 4;       // float [2][4]: the quarters' decays
    static constexpr uint32_t bar = dec + 32;           // A; O1; D; O2; loads of Q and K; of V
    static constexpr uint32_t misc = bar + 48;          // tensor-memory address
    static constexpr uint32_t bytes = misc + 8;
};
static_assert(2 * (TcSmem<128>::bytes + 128 + 1024) <= 228 * 1024 && TcSmem<64>::bytes <= TcSmem<128>::bytes, "two blocks on an SM");

// Zeroes the rows [n, 128) of `blocks` tiles.
__device__ __forceinline__ void tc_clear_rows(unsigned char* sm, int blocks, int n) {
    for (int b = 0; b < blocks; ++b)
        for (uint32_t o = n * 128 + threadIdx.x * 16; o < kTileBytes; o += kTcThr * 16)
            *reinterpret_cast<uint4*>(sm + b * kTileBytes + o) = make_uint4(0, 0, 0, 0);
}

struct TcMaps {  // 3-D maps {channels, heads, rows}; y: the forward's output, or its gradient
    CUtensorMap q, k, v, y;
};
// Eight 32-bit values, 32-byte aligned: a whole sector in one store.
__device__ __forceinline__ void store_32(void* p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :
                 : "l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// 16 packed bf16 values to a row's columns c .. c + 15, of which those before `cols` (a multiple of 8) exist.
__device__ __forceinline__ void store_row16(__nv_bfloat16* p, const uint32_t (&v)[8], int c, int cols, bool wide) {
    if (wide) {  // rows start on 32 bytes
        if (c < cols) store_32(p, v);
    } else {
        if (c < cols) *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[2], v[3]);
        if (c + 8 < cols) *reinterpret_cast<uint4*>(p + 8) = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// Quarters whose decays rise are marked by the sign of their decay, as every thread reads those of all quarters.
__device__ __forceinline__ float mark_rise(float decay, float g) { return __any_sync(0xffffffffu, g > kRise) ? -decay : decay; }
__device__ __forceinline__ bool any_rise(const float4& e) {
    return __any_sync(0xffffffffu, (__float_as_int(e.x) | __float_as_int(e.y) | __float_as_int(e.z) | __float_as_int(e.w)) < 0);
}
// Such a chunk's scores of this warp's rows and of two quarters of columns take their weights where they lie.
__device__ __noinline__ void weigh_scores(uint32_t lanes, int grp, int q, Exponent own, const float* g, long long step, int n) {
#pragma unroll 1
    for (int e = min(grp + 2, q + 1); grp < e; ++grp) {
        const Exponent at = chunk_sum(g, step, n, grp).at;
#pragma unroll 1
        for (int c = 0; c < 32; c += 16) {
            float a[16];
            uint32_t w[16];
            tc::ld16(lanes + 32 * grp + c, a);
            tc::wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const Exponent e{__shfl_sync(0xffffffffu, at.hi, c + j), __shfl_sync(0xffffffffu, at.lo, c + j)};
                w[j] = __float_as_uint(a[j] * decay_between(own, e));
            }
            tc::st16(lanes + 32 * grp + c, w);
        }
    }
    tc::wait_st();
}

template <int DK, bool OUT>
__global__ void __launch_bounds__(kTcThr, 2)
tc_forward_kernel(const __grid_constant__ TcMaps maps, Shape sh, PackedPlan plan, Tensors x, const float* start, float* st_loc,
                  float* piece_decay, unsigned* status) {
    extern __shared__ __align__(1024) unsigned char smem[];
    using M = TcSmem<DK>;
    float* s_u = reinterpret_cast<float*>(smem + M::u);
    float* s_dec = reinterpret_cast<float*>(smem + M::dec);
    unsigned long long* bar = reinterpret_cast<unsigned long long*>(smem + M::bar);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + M::misc);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), q = warp & 3, half = warp >> 2;
    Piece pc;
    const int tiles = (sh.dv + kTile - 1) / kTile, per = sh.H * tiles, hy = blockIdx.x % per;
    int id;
    if (!get_piece(sh, plan, blockIdx.x / per, pc, id)) return wait_for_primary();  // no launch ends before those it overlaps
    // a piece's own state is needed where another follows, or where its sequence's final state is asked for;
    // a sequence of one piece carries its state alone
    if (!OUT && (pc.flags == 3 || ((pc.flags & 2) && (!x.st || sh.look_back)))) return;
    const bool exact = x.st && (!OUT || (sh.look_back ? (pc.flags & 2) : pc.flags == 3));
    const int h = hy / tiles, c0 = (hy - h * tiles) * kTile;
    const int hk = key_head(sh, h), cols = min(kTile, sh.dv - c0);
    const uint32_t base = smem_u32(smem);

    if (warp == 0) tc::alloc(s_tmem, 256);
    if (tid == 0) {
        for (int i = 0; i < 6; ++i) mbar_init(bar + i, 1);
        fence_mbar_init();
    }
    __syncthreads();
    // The outputs' blocks may begin with what needs no state.  Only now: they take tensor memory and wait for
    // this block, which must have its own by then.
    if (!OUT) launch_dependents();
    constexpr int blocks = M::kBlocks;
    // by one thread; Q and K complete on one barrier, whose bytes the first of the two announces
    auto load_q = [&](int t0) {
        for (int b = 0; b < blocks; ++b) tc::load_tile(smem + M::q + b * kTileBytes, &maps.q, 64 * b, hk, pc.row + t0, bar + 4);
    };
    auto load_k = [&](int t0) {
        for (int b = 0; b < blocks; ++b) tc::load_tile(smem + M::k + b * kTileBytes, &maps.k, 64 * b, hk, pc.row + t0, bar + 4);
    };
    auto announce = [&]() { mbar_arrive_expect_tx(bar + 4, (OUT ? 2 : 1) * blocks * kTileBytes); };
    auto load_v = [&](int t0) {
        mbar_arrive_expect_tx(bar + 5, kTileBytes);
        tc::load_tile(smem + M::v, &maps.v, c0, h, pc.row + t0, bar + 5);
    };
    const float* gg = x.g + (sh.head_decay ? h : (long long)pc.row * sh.gs + h);
    auto load_g = [&](int t0) -> float {  // this lane's token of its quarter
        const int t = t0 + 32 * q + lane;
        return t < pc.len ? __ldg(gg + (sh.head_decay ? 0 : (long long)t * sh.gs)) : 0.f;
    };
    // Local sums of the quarter: own exponent and its power, the row factor for the own quarter (negative:
    // each pair by itself), and the quarter's decay and column weights in shared memory.
    Exponent own;
    float own_pow, own_diag;
    auto scan_g = [&](float g, int parity) {
        const WarpSums w = warp_sums(g);
        const float nan = __int_as_float(0x7fffffff);
        own = w.own;
        own_pow = w.bad ? nan : ex2_approx(own.hi + own.lo);
        own_diag = w.total.hi > -100.f && !w.bad ? ex2_approx(-w.to_end) : -1.f;
        if (w.bad) own.lo = nan;
        if (half == 0) {
            s_u[32 * q + lane] = w.bad ? nan : ex2_approx(w.to_end);
            const float d = mark_rise(decay_of(w.total), g);
            if (lane == 0) s_dec[4 * parity + q] = w.bad ? nan : d;
        }
    };
    float g_next = load_g(0);

    const uint32_t lead = warp == 0 ? tc::elect_one() : 0;  // the thread that issues products and copies
    if (lead && pc.len > 0) {
        announce();
        if (OUT) load_q(0);
        load_k(0);
        load_v(0);
    }
    if (OUT && pc.flags != 3) wait_for_primary();

    // state rows: dk 128: row 32 q + lane; dk 64: the accumulator of an M = 64 product uses the first 16
    // lanes of each quarter
    const int srow = DK == 128 ? 32 * q + lane : 16 * q + lane;
    const bool sact = DK == 128 || lane < 16;
    float2 S[16];
    {
        const size_t at = ((size_t)id * sh.H + h) * sh.dk * sh.dv;
        const float* s_in = !OUT ? nullptr : pc.flags != 3 ? start + at
                            : x.s0 ? x.s0 + ((size_t)pc.seq * sh.H + h) * sh.dk * sh.dv : nullptr;
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            const int c = 32 * half + 2 * j;
            if (sact && srow < sh.dk && c < cols) {
                const size_t o = (size_t)srow * sh.dv + c0 + c;
                if (OUT && sh.look_back && pc.flags != 3) v = look_back(sh, start, piece_decay, x.s0, id, pc.seq, h, o);
                else if (s_in) v = __ldcg(reinterpret_cast<const float4*>(s_in + o));
            }
            S[j] = make_float2(v.x, v.y);
            S[j + 1] = make_float2(v.z, v.w);
        }
    }
    auto put_state = [&]() {
        if (sact) {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2 z = S[4 * v + j];
                    hi[j] = tc::take_part(z);
                    lo[j] = pack2<__nv_bfloat16>(z.x, z.y);
                }
                const uint32_t o = tc::swz(srow, 4 * half + v);
                *reinterpret_cast<uint4*>(smem + M::s + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(smem + M::slo + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        }
    };
    if (OUT) put_state();
    scan_g(g_next, 0);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *s_tmem;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
    const uint32_t cA = tmem, cO2 = tmem, cP = tmem + 64, cO1 = tmem + 128, cD = tmem + 192;
    const uint64_t dQ = tc::desc(base + M::q, 0), dK = tc::desc(base + M::k, 0), dKt = tc::desc(base + M::k, kTileBytes),
                   dV = tc::desc(base + M::v, 0), dVhi = tc::desc(base + M::vhi, 0), dVmid = tc::desc(base + M::vmid, 0),
                   dVlo = tc::desc(base + M::vlo, 0), dShi = tc::desc(base + M::s, 0), dSlo = tc::desc(base + M::slo, 0);
    bool ok = true;
    float decay = 1.f;
    int c = 0;
    for (int t0 = 0; t0 < pc.len; t0 += kTcC, ++c) {
        const int par = c & 1;
        const bool more = t0 + kTcC < pc.len;
        ok = tc::wait(bar + 4, par);
        if (pc.len - t0 < kTcC) {  // rows of the next sequence
            ok = tc::wait(bar + 5, par) && ok;
            tc_clear_rows(smem + M::k, blocks, pc.len - t0);
            tc_clear_rows(smem + M::v, 1, pc.len - t0);
        }
        fence_proxy_async_smem();
        tc::fence_before();
        if (!__syncthreads_and(ok)) break;
        if (warp == 0) {
            tc::fence_after();
            if (OUT) {
                constexpr uint32_t iA = tc::idesc(128, 128, false, false), iO = tc::idesc(128, 64, false, true);
                const int nk = (sh.dk + 15) / 16;
#pragma unroll
                for (int k = 0; k < DK / 16; ++k) {  // 16 channels: 32 bytes inside a row, four steps per 64-column block
                    const uint32_t o = (k >> 2) * kTileBytes + (k & 3) * 32;
                    if (k < nk) tc::mma_ss(cA, tc::ahead(dQ, o), tc::ahead(dK, o), iA, k > 0, lead);
                }
                tc::commit(bar, lead);
                // the small parts first, here and below: an accumulator drops what lies behind its last bit, at
                // every step and to one side, and is small itself until the large part comes
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k) {
                        const uint32_t o = (k >> 2) * kTileBytes + (k & 3) * 32;
                        if (k < nk) tc::mma_ss(cO1, tc::ahead(dQ, o), tc::ahead(part ? dShi : dSlo, k * 2048), iO, part + k > 0, lead);
                    }
                tc::commit(bar + 1, lead);
            }
        }
        g_next = load_g(t0 + kTcC);
        float4 E = *reinterpret_cast<const float4*>(s_dec + 4 * par);
        const bool rises = any_rise(E);
        const long long step = sh.head_decay ? 0 : sh.gs;
        float all = 1.f;
        if (rises) {  // sums and powers of the whole chunk in place of the quarter's
            const ChunkSum s = chunk_sum(gg + t0 * step, step, pc.len - t0, q);
            own = s.at;
            own_pow = decay_of(own);
            if (half == 0) s_u[32 * q + lane] = decay_behind(own, s.total);
            E = make_float4(1.f, 1.f, 1.f, 1.f);
            all = decay_of(s.total);
            __syncthreads();
        }
        const float E23 = E.z * E.w, E123 = E.y * E23, chunk = all * (E.x * E123);
        const float head = sh.scale * own_pow * (q > 0 ? E.x : 1.f) * (q > 1 ? E.y : 1.f) * (q > 2 ? E.z : 1.f);
        if (!OUT) decay *= chunk;
        ok = tc::wait(bar + 5, par);
        if (OUT && DK == 128) ok = tc::wait(bar + 1, par) && ok;  // Q and S, which V~ replaces, have been read
        // weighted v: e^{G_C - G_j} = u_j times the decays of the quarters behind j's
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (tid >> 3) + 32 * i;  // quarter i
            const uint32_t o = tc::swz(r, tid & 7);
            const uint4 v = *reinterpret_cast<const uint4*>(smem + M::v + o);
            const float w = s_u[r] * (i == 0 ? E123 : i == 1 ? E23 : i == 2 ? E.w : 1.f);
            const float2 w2 = make_float2(w, w);
            const uint32_t in[4] = {v.x, v.y, v.z, v.w};
            uint32_t part[4];
            float2 z[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                z[j] = tc::mul2(unpack2<__nv_bfloat16>(in[j]), w2);
                part[j] = pack2<__nv_bfloat16>(z[j].x, z[j].y);
            }
            *reinterpret_cast<uint4*>(smem + M::vhi + o) = make_uint4(part[0], part[1], part[2], part[3]);
            if (exact) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    z[j] = tc::sub2(z[j], unpack2<__nv_bfloat16>(part[j]));
                    part[j] = tc::take_part(z[j]);
                }
                *reinterpret_cast<uint4*>(smem + M::vmid + o) = make_uint4(part[0], part[1], part[2], part[3]);
                *reinterpret_cast<uint4*>(smem + M::vlo + o) =
                    make_uint4(pack2<__nv_bfloat16>(z[0].x, z[0].y), pack2<__nv_bfloat16>(z[1].x, z[1].y),
                               pack2<__nv_bfloat16>(z[2].x, z[2].y), pack2<__nv_bfloat16>(z[3].x, z[3].y));
            }
        }
        fence_proxy_async_smem();
        tc::fence_before();
        if (!__syncthreads_and(ok)) break;
        if (warp == 0) {
            tc::fence_after();
            constexpr uint32_t iD = tc::idesc(DK, 64, true, true);
#pragma unroll
            for (int part = 0; part < 3; ++part) {
                if (part == 2 || exact)
#pragma unroll
                    for (int k = 0; k < kTcC / 16; ++k)
                        tc::mma_ss(cD, tc::ahead(dKt, k * 2048), tc::ahead(part == 2 ? dVhi : part ? dVmid : dVlo, k * 2048), iD,
                                   k > 0 || (part > 0 && exact), lead);
            }
            tc::commit(bar + 2, lead);
        }
        if constexpr (OUT) {
            ok = tc::wait(bar, par);
            tc::fence_after();
            // Up to 64 tokens fill half of P: the other half takes what bf16 leaves of them, for the few scores of
            // a short prompt are its outputs' only factors, and their roundings do not average out.
            const bool brief = pc.len - t0 <= kTcC / 2, rest = brief && half;
            if (rises) {
                if (!rest) weigh_scores(lanes, brief ? 0 : 2 * half, q, own, gg + t0 * step, step, pc.len - t0);
                own_pow = own_diag = 1.f;
                if (half == 0) s_u[32 * q + lane] = 1.f;
                tc::fence_before();
                __syncthreads();
                tc::fence_after();
            }
            uint32_t p[2][16];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int grp = (brief ? 0 : 2 * half) + i;
                if (grp > q) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) p[i][j] = 0u;
                } else {
                    float a[32];
                    tc::ld32(lanes + 32 * grp, a);
                    tc::wait_ld();
                    if (grp < q || own_diag >= 0.f) {
                        // the row's factor; between two quarters, those between decay too
                        const float f = sh.scale * (grp < q ? own_pow * (grp < 1 && q > 1 ? E.y : 1.f) * (grp < 2 && q > 2 ? E.z : 1.f) : own_diag);
                        const float2 f2 = make_float2(f, f);
                        const float4* u4 = reinterpret_cast<const float4*>(s_u + 32 * grp);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float4 w = u4[j];
                            const float2 a0 = tc::mul2(make_float2(a[4 * j], a[4 * j + 1]), tc::mul2(f2, make_float2(w.x, w.y)));
                            const float2 a1 = tc::mul2(make_float2(a[4 * j + 2], a[4 * j + 3]), tc::mul2(f2, make_float2(w.z, w.w)));
                            a[4 * j] = a0.x, a[4 * j + 1] = a0.y, a[4 * j + 2] = a1.x, a[4 * j + 3] = a1.y;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            Exponent e;
                            e.hi = __shfl_sync(0xffffffffu, own.hi, j);
                            e.lo = __shfl_sync(0xffffffffu, own.lo, j);
                            a[j] *= sh.scale * decay_between(own, e);
                        }
                    }
                    if (rest) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) a[j] -= __bfloat162float(__float2bfloat16_rn(a[j]));
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) p[i][j] = pack2<__nv_bfloat16>(a[2 * j], a[2 * j + 1]);
                    if (grp == q) {  // later tokens of the quarter, whatever stands there
#pragma unroll
                        for (int j = 0; j < 16; ++j) p[i][j] &= lane > 2 * j ? 0xffffffffu : lane == 2 * j ? 0xffffu : 0u;
                    }
                }
            }
            // P's columns lie over scores that the quarter's other warp reads
            tc::fence_before();
            asm volatile("bar.sync %0, 64;" : : "r"(1 + q) : "memory");
            tc::fence_after();
            tc::st16(lanes + 64 + 32 * half, p[0]);
            tc::st16(lanes + 64 + 32 * half + 16, p[1]);
            tc::wait_st();
            tc::fence_before();
            if (!__syncthreads_and(ok)) break;
            if (warp == 0) {
                tc::fence_after();
                constexpr uint32_t iO = tc::idesc(128, 64, false, true);
#pragma unroll
                for (int k = 0; k < kTcC / 16; ++k)
                    tc::mma_ts(cO2, cP + 8 * k, tc::ahead(dV, (k & (brief ? 3 : 7)) * 2048), iO, k > 0, lead);
                tc::commit(bar + 3, lead);
            }
        }
        ok = tc::wait(bar + 2, par);  // D, and every product before it
        tc::fence_after();
        if (lead && ok && more) {
            announce();
            if (OUT) load_q(t0 + kTcC);
            load_k(t0 + kTcC);
            if (!OUT) load_v(t0 + kTcC);
        }
        {
            float d[32];
            tc::ld32(lanes + 192 + 32 * half, d);
            tc::wait_ld();
            const float2 c2 = make_float2(chunk, chunk);
#pragma unroll
            for (int j = 0; j < 16; ++j) S[j] = tc::fma2(c2, S[j], make_float2(d[2 * j], d[2 * j + 1]));
        }
        if constexpr (OUT) {
            put_state();
            ok = tc::wait(bar + 3, par) && ok;
            tc::fence_after();
            if (DK == 64 && lead && ok && more) load_v(t0 + kTcC);
            const int row = 32 * q + lane;
            const bool in = t0 + row < pc.len;
            __nv_bfloat16* y = (__nv_bfloat16*)x.y + ((size_t)(pc.row + t0 + row) * sh.H + h) * sh.dv + c0 + 32 * half;
            const float2 h2 = make_float2(head, head);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float a[16], b[16];
                tc::ld16(lanes + 128 + 32 * half + 16 * j, a);
                tc::ld16(lanes + 32 * half + 16 * j, b);
                tc::wait_ld();
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 z = tc::fma2(h2, make_float2(a[2 * i], a[2 * i + 1]), make_float2(b[2 * i], b[2 * i + 1]));
                    o[i] = pack2<__nv_bfloat16>(z.x, z.y);
                }
                // a whole chunk leaves through a tile in one TMA store, 128 bytes a row; the piece's last one,
                // whose rows may end, from here
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 w = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    if (more) *reinterpret_cast<uint4*>(smem + M::y + tc::swz(row, 4 * half + 2 * j + i)) = w;
                    else if (in && 32 * half + 16 * j + 8 * i < cols) *reinterpret_cast<uint4*>(y + 16 * j + 8 * i) = w;
                }
            }
            if (more) {
                fence_proxy_async_smem();
                tc::fence_before();
                if (!__syncthreads_and(ok)) break;
                if (lead) tc::store_tile(&maps.y, smem + M::y, c0, h, pc.row + t0);
            }
        }
        scan_g(g_next, par ^ 1);
        if (OUT && lead && more) {  // y's tile is free again for what comes next
            tc::store_read();
            if (DK == 128) load_v(t0 + kTcC);
        }
    }
    if (!ok) set_status(status, kStatusTimeout);
    float* s_out = !OUT ? st_loc + ((size_t)id * sh.H + h) * sh.dk * sh.dv
                   : exact ? x.st + ((size_t)pc.seq * sh.H + h) * sh.dk * sh.dv : nullptr;
    if (s_out && sact && srow < sh.dk) {
#pragma unroll
        for (int j = 0; j < 16; j += 2)
            if (32 * half + 2 * j < cols)
                *reinterpret_cast<float4*>(s_out + (size_t)srow * sh.dv + c0 + 32 * half + 2 * j) =
                    make_float4(S[j].x, S[j].y, S[j + 1].x, S[j + 1].y);
    }
    if (!OUT && tid == 0 && c0 == 0) piece_decay[(size_t)id * sh.H + h] = decay;
    if (OUT && lead) tc::store_done();
    if (OUT && pc.flags == 3) wait_for_primary();  // no launch ends before those it overlaps
    tc::fence_before();
    __syncthreads();
    if (warp == 0) tc::dealloc(tmem, 256);
}

}  // namespace la
}  // namespace fv
