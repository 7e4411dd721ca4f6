// fv_linattn_tc_grad.cuh -- the bf16 gradient of linear attention on the 5th-generation tensor cores.
//
// Chunks of 128 tokens, all at once: (1) each chunk's own states, (2) the joining pass turns them into
// the states entering and the state gradients leaving each chunk, (3) the gradients of one chunk and head
// per block.  In (3), with token i the later and j the earlier one of a pair:
//   tensor cores:  A' = K Q^T, X' = V dY^T                    (rows j, columns i; X' over all tiles of v)
//   threads:       A = w A' (bf16, tensor memory), P = w X' (bf16, registers), M = w A' X'  -> dg
//   per 64 columns of v:  dv1 = K dS, dq1 += dY S^T, dk1 += V dS^T, then dv2 = A dY
//   threads:       dv = e^{G_C - G_j} dv1 + dv2;  P into shared memory, over V and dY
//   tensor cores:  dk2 = P Q (P as stored), dq2 = P^T K (the same tile read the other way)
//   threads:       dq = scale e^{G_i} dq1 + dq2, dk = e^{G_C - G_j} dk1 + dk2, and dg.
// Weighted scores are rounded to bf16 as in the forward.  States go in as three bf16 parts where the
// result feeds dg (dq1, dk1), as two in dv1; M is the product of fp32 accumulators.  So dg and the states'
// gradients, which are returned in fp32, are exact to fp32's order.
//
// 8 x 4096 tokens x 12 heads of 64 x 64: (1) 80 us, (2) 29 us, (3) 175 us each by itself, 283 us
// together, as a launch begins while the one before it ends; the traffic of the arguments alone
// would take 54 us.  (1) and (2) are bound by the states, written and read several times (100 MB each); (3) by
// the threads' work between the products and the waits for them, at two blocks on an SM (128 registers).
#pragma once

#include "fv_linattn_simt.cuh"
#include "fv_linattn_tc.cuh"

namespace fv {
namespace la {

// Local sums of this lane's quarter (see fv_linattn_tc.cuh): the weights u = exp2(T - L) and, of the other
// direction, hl = exp2(L), and the quarter's decay (and its exponent), into shared memory; own exponent and, for pairs inside
// the quarter, exp2(-L) (negative: each pair by itself).
struct TcScan {
    Exponent own;
    float pow, diag;
};
__device__ __forceinline__ TcScan tc_scan(float g, int lane, int q, bool write, float* u, float* hl, float* dec, float* tot) {
    const WarpSums w = warp_sums(g);
    const float nan = __int_as_float(0x7fffffff);
    TcScan r;
    r.own = w.own;
    r.pow = w.bad ? nan : power_of(w.own.hi, w.own.lo);
    r.diag = w.total.hi > -100.f && !w.bad ? power_of(-w.own.hi, -w.own.lo) : -1.f;
    if (w.bad) r.own.lo = nan;
    if (write) {
        u[32 * q + lane] = w.bad ? nan : ex2_approx(w.to_end);
        hl[32 * q + lane] = r.pow;
        const float d = mark_rise(decay_of(w.total), g);
        if (lane == 0) {
            dec[q] = w.bad ? nan : d;
            if (tot) tot[2 * q] = w.total.hi, tot[2 * q + 1] = w.bad ? nan : w.total.lo;
        }
    }
    return r;
}

// ---- the chunks' own states ---------------------------------------------------------------------------
template <int DK>
struct TcLocalSmem {
    static constexpr uint32_t a = 0;                                // K or Q
    static constexpr uint32_t b = a + DK / 64 * kTileBytes;         // V or dY, then its weighted form's three parts in turn
    static constexpr uint32_t u = b + kTileBytes;                   // float [2][128]
    static constexpr uint32_t dec = u + 2 * kTcC * 4;               // float [4]
    static constexpr uint32_t bar = dec + 16;                       // products; loads
    static constexpr uint32_t misc = bar + 16;
    static constexpr uint32_t bytes = misc + 8;
};

// One block per (chunk, head, 64 columns of v), four on an SM (blocks that walk several with the next one's
// loads in flight take 76 us for 80 us of the case above, but 11 us more for 6 heads of 128).  blockIdx.z 0: S = sum_j e^{G_C - G_j} k_j v_j^T and the
// chunk's decay, 1: dS = scale sum_i e^{G_i} q_i dy_i^T.
template <int DK>
__global__ void __launch_bounds__(kTcThr, 4)
tc_local_kernel(const __grid_constant__ TcMaps maps, Shape sh, PackedPlan plan, Tensors x, float* __restrict__ S, float* __restrict__ dS, float* __restrict__ decay,
                unsigned* status) {
    extern __shared__ __align__(1024) unsigned char smem[];
    using M = TcLocalSmem<DK>;
    float* s_u = reinterpret_cast<float*>(smem + M::u);
    float* s_dec = reinterpret_cast<float*>(smem + M::dec);
    unsigned long long* bar = reinterpret_cast<unsigned long long*>(smem + M::bar);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + M::misc);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), q = warp & 3, half = warp >> 2;
    const bool grad = blockIdx.z == 1;
    Piece pc;
    int id;
    if (!get_piece(sh, plan, blockIdx.x, pc, id)) return;
    const int tiles = (sh.dv + kTile - 1) / kTile;
    const int h = blockIdx.y / tiles, c0 = (blockIdx.y - h * tiles) * kTile;
    const int hk = key_head(sh, h), cols = min(kTile, sh.dv - c0), t = 32 * q + lane;
    const long long step = sh.head_decay ? 0 : sh.gs;
    const float* first = x.g + pc.row * step + h;
    const float g = t < pc.len ? __ldg(first + t * step) : 0.f;
    const uint32_t base = smem_u32(smem);
    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_init(bar + 1, 1);
        fence_mbar_init();
        if (pc.len > 0) {
            mbar_arrive_expect_tx(bar + 1, (DK / 64 + 1) * kTileBytes);
            for (int i = 0; i < DK / 64; ++i) tc::load_tile(smem + M::a + i * kTileBytes, grad ? &maps.q : &maps.k, 64 * i, hk, pc.row, bar + 1);
            tc::load_tile(smem + M::b, grad ? &maps.y : &maps.v, c0, h, pc.row, bar + 1);
        }
    }
    if (warp == 0) tc::alloc(s_tmem, 64);
    tc_scan(g, lane, q, half == 0, s_u, s_u + kTcC, s_dec, nullptr);
    tc::fence_before();
    __syncthreads();
    launch_dependents();  // behind its own tensor memory, as in the forward
    tc::fence_after();
    const uint32_t tmem = *s_tmem;
    bool ok = pc.len == 0 || tc::wait(bar + 1, 0);
    if (pc.len < kTcC) {  // rows of the next sequence
        tc_clear_rows(smem + M::a, DK / 64, pc.len);
        tc_clear_rows(smem + M::b, 1, pc.len);
        __syncthreads();
    }
    float4 E = *reinterpret_cast<const float4*>(s_dec);
    float chunk = (E.x * E.y) * (E.z * E.w);
    if (any_rise(E)) {  // sums and powers of the whole chunk in place of the quarter's
        const ChunkSum s = chunk_sum(first, step, pc.len, q);
        if (half == 0) s_u[t] = decay_behind(s.at, s.total), s_u[kTcC + t] = decay_of(s.at);
        E = make_float4(1.f, 1.f, 1.f, 1.f);
        chunk = decay_of(s.total);
        __syncthreads();
    }
    if (tid == 0 && c0 == 0 && !grad) decay[(size_t)id * sh.H + h] = chunk;
    // Three parts of the weighted rows, one after the other through b: the rows stay in registers as they came,
    // so the tiles are small enough for four blocks on an SM, whose load latency is what bounds the kernel.
    uint4 v[4];
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (tid >> 3) + 32 * i;  // quarter i
        const float far = grad ? sh.scale * (i > 0 ? E.x : 1.f) * (i > 1 ? E.y : 1.f) * (i > 2 ? E.z : 1.f)
                               : (i < 1 ? E.y : 1.f) * (i < 2 ? E.z : 1.f) * (i < 3 ? E.w : 1.f);
        w[i] = s_u[(grad ? kTcC : 0) + r] * far;
        v[i] = *reinterpret_cast<const uint4*>(smem + M::b + tc::swz(r, tid & 7));
    }
    const uint64_t dA = tc::desc(base + M::a, kTileBytes), dB = tc::desc(base + M::b, 0);
    const uint32_t lead = warp == 0 ? tc::elect_one() : 0;
#pragma unroll
    for (int turn = 0; turn < 3; ++turn) {
        const int part = 2 - turn;  // the small parts first
        if (turn) ok = tc::wait(bar, (turn - 1) & 1) && ok;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t in[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 z = tc::mul2(unpack2<__nv_bfloat16>(in[j]), make_float2(w[i], w[i]));
#pragma unroll
                for (int p = 0; p < part; ++p) tc::take_part(z);
                o[j] = pack2<__nv_bfloat16>(z.x, z.y);
            }
            *reinterpret_cast<uint4*>(smem + M::b + tc::swz((tid >> 3) + 32 * i, tid & 7)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (warp == 0) {
            tc::fence_after();
            constexpr uint32_t id = tc::idesc(DK, 64, true, true);
#pragma unroll
            for (int k = 0; k < kTcC / 16; ++k)
                tc::mma_ss(tmem, tc::ahead(dA, k * 2048), tc::ahead(dB, k * 2048), id, turn + k > 0, lead);
            tc::commit(bar, lead);
        }
    }
    ok = tc::wait(bar, 0) && ok;  // the third phase
    if (!ok) set_status(status, kStatusTimeout);
    tc::fence_after();
    const int row = DK == 128 ? 32 * q + lane : 16 * q + lane;  // as the forward's state rows
    float d[32];
    tc::ld32(tmem + ((uint32_t)(32 * q) << 16) + 32 * half, d);
    tc::wait_ld();
    if (ok && (DK == 128 || lane < 16) && row < sh.dk) {
        float* out = (grad ? dS : S) + (((size_t)id * sh.H + h) * sh.dk + row) * sh.dv + c0 + 32 * half;
#pragma unroll
        for (int j = 0; j < 32; j += 8)  // dv is a multiple of 8: every group of 8 starts on 32 bytes
            if (32 * half + j < cols) {
                uint32_t v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(d[j + i]);
                store_32(out + j, v);
            }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) tc::dealloc(tmem, 64);
}

// ---- one chunk's gradients --------------------------------------------------------------------------
template <int DK>
struct TcGradSmem {
    static constexpr uint32_t kBlocks = DK / 64;
    static constexpr uint32_t q = 0;                         // Q; between the scores and dk2 third parts of S, dS
    static constexpr uint32_t k = q + kBlocks * kTileBytes;
    static constexpr uint32_t v = k + kBlocks * kTileBytes;  // V and dY; P in the end
    static constexpr uint32_t y = v + kTileBytes;
    static constexpr uint32_t s = y + kTileBytes;            // S hi, S lo, dS hi, dS lo: DK rows of 64 columns
    static constexpr uint32_t kS = DK * 128;
    static constexpr uint32_t u = s + 4 * kS;                // float [128]
    static constexpr uint32_t hl = u + kTcC * 4;             // float [128]
    static constexpr uint32_t col = hl + kTcC * 4;           // float [4][128]: column sums of M by quarter of rows
    static constexpr uint32_t row = col + 4 * kTcC * 4;      // float [4][128]: row sums of M by group of columns
    static constexpr uint32_t inq = row + 4 * kTcC * 4;      // float [2][128]
    static constexpr uint32_t outk = inq + 2 * kTcC * 4;     // float [2][128]
    static constexpr uint32_t dec = outk + 2 * kTcC * 4;     // float [4]: the quarters' decays
    static constexpr uint32_t tot = dec + 16;                // float [4][2]: their exponents
    static constexpr uint32_t sums = tot + 32;               // float [4][4], [2][4], [2][4]: row, inq, outk by quarter
    static constexpr uint32_t red = sums + 128;              // float [8]
    static constexpr uint32_t bar = red + 32;                // products; loads
    static constexpr uint32_t misc = bar + 16;
    static constexpr uint32_t bytes = misc + 8;
};
static_assert(2 * (TcGradSmem<64>::bytes + 128 + 1024) <= 228 * 1024, "two blocks on an SM");
static_assert(TcGradSmem<128>::bytes <= 227 * 1024, "one block on an SM");

__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// v[c] of lane l summed over the lanes: lane c returns the sum of column c.  31 exchanges.
__device__ __forceinline__ float lane_columns(float (&v)[32], int lane) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int c = 0; c < 16; ++c)
            if (c < o) {
                const float give = up ? v[c] : v[c + o], keep = up ? v[c + o] : v[c];
                v[c] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
    }
    return v[0];
}

// Of this lane's row and the 32 columns of a group, m (zero where there is no pair): the row's sum, its sum over the
// warp's rows, and for each column what of the rows lies at or behind it (behind it in their own quarter).
__device__ __forceinline__ void pair_sums(float (&m)[32], int grp, int q, int lane, float* s_row, float* s_col, float* s_sum) {
    // what of this row lies at or behind column t of the group: sums inside eights, then across them
#pragma unroll
    for (int j = 6; j >= 0; --j)
#pragma unroll
        for (int o = 0; o < 32; o += 8) m[o + j] += m[o + j + 1];
#pragma unroll
    for (int o = 16; o >= 0; o -= 8)
#pragma unroll
        for (int j = 7; j >= 0; --j) m[o + j] += m[o + 8];
    s_row[grp * kTcC + 32 * q + lane] = m[0];
    {
        const float z = warp_total(m[0]);
        if (lane == 0) s_sum[4 * grp + q] = z;
    }
    if (grp == q)
#pragma unroll
        for (int j = 0; j < 32; ++j) m[j] = j > lane ? m[j] : 0.f;
    s_col[q * kTcC + 32 * grp + lane] = lane_columns(m, lane);
}

// The scores of a chunk whose decays rise (see fv_linattn_tc.cuh), of this warp's rows and of two groups of columns, take
// their weights where they lie; dg's sums over their products, here too.
__device__ __noinline__ void weigh_pairs(uint32_t sa, uint32_t sx, int grp, int q, Exponent own, const float* g, long long step, int n,
                                         float scale, float* s_row, float* s_col, float* s_sum) {
    const int lane = threadIdx.x & 31, end = grp + 2;
#pragma unroll 1
    for (grp = max(grp, q); grp < end; ++grp) {
        const Exponent at = chunk_sum(g, step, n, grp).at;
        float m[32];
#pragma unroll
        for (int c = 0; c < 32; c += 16) {
            float a[16], b[16];
            uint32_t wa[16], wb[16];
            tc::ld16(sa + 32 * grp + c, a);
            tc::ld16(sx + 32 * grp + c, b);
            tc::wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float w = decay_between(Exponent{__shfl_sync(0xffffffffu, at.hi, c + j), __shfl_sync(0xffffffffu, at.lo, c + j)}, own);
                wa[j] = __float_as_uint(a[j] * w);
                wb[j] = __float_as_uint(b[j] * w);
                m[c + j] = grp > q || c + j >= lane ? scale * (a[j] * w) * b[j] : 0.f;
            }
            tc::st16(sa + 32 * grp + c, wa);
            tc::st16(sx + 32 * grp + c, wb);
        }
        pair_sums(m, grp, q, lane, s_row, s_col, s_sum);
    }
    tc::wait_st();
}

template <int DK>
__global__ void __launch_bounds__(kTcThr, DK == 64 ? 2 : 1)
tc_grad_kernel(const __grid_constant__ TcMaps maps, Shape sh, PackedPlan plan, Tensors x, const float* S_in, const float* dS_out, GradOut out,
               unsigned* status) {
    extern __shared__ __align__(1024) unsigned char smem[];
    using M = TcGradSmem<DK>;
    constexpr uint32_t kCols = DK == 64 ? 256 : 512;
    float* s_u = reinterpret_cast<float*>(smem + M::u);
    float* s_hl = reinterpret_cast<float*>(smem + M::hl);
    float* s_col = reinterpret_cast<float*>(smem + M::col);
    float* s_row = reinterpret_cast<float*>(smem + M::row);
    float* s_in = reinterpret_cast<float*>(smem + M::inq);
    float* s_out = reinterpret_cast<float*>(smem + M::outk);
    float* s_dec = reinterpret_cast<float*>(smem + M::dec);
    float* s_tot = reinterpret_cast<float*>(smem + M::tot);
    float* s_sum = reinterpret_cast<float*>(smem + M::sums);
    float* s_red = reinterpret_cast<float*>(smem + M::red);
    unsigned long long* bar = reinterpret_cast<unsigned long long*>(smem + M::bar);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + M::misc);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), q = warp & 3, half = warp >> 2;
    Piece pc;
    int id;
    if (!get_piece(sh, plan, blockIdx.x, pc, id)) return wait_for_primary();
    const int h = blockIdx.y, hk = key_head(sh, h), n = pc.len;
    if (n == 0) {
        wait_for_primary();  // no launch ends before those it overlaps
        if (sh.head_decay && tid == 0) out.dg[(size_t)id * sh.H + h] = 0.f;
        return;
    }
    const int tok = 32 * q + lane;  // this thread's token (rows i and j alike)
    const long long step = sh.head_decay ? 0 : sh.gs;
    const float* first = x.g + pc.row * step + h;
    const float g = tok < n ? __ldg(first + tok * step) : 0.f;
    const int tiles = (sh.dv + kTile - 1) / kTile;
    const uint32_t base = smem_u32(smem);
    const size_t state_at = ((size_t)id * sh.H + h) * sh.dk * sh.dv;
    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_init(bar + 1, 1);
        fence_mbar_init();
    }
    __syncthreads();
    const uint32_t lead = warp == 0 ? tc::elect_one() : 0;  // the thread that issues products and loads
    auto load_vy = [&](int t) {
        mbar_arrive_expect_tx(bar + 1, 2 * kTileBytes);
        tc::load_tile(smem + M::v, &maps.v, t * kTile, h, pc.row, bar + 1);
        tc::load_tile(smem + M::y, &maps.y, t * kTile, h, pc.row, bar + 1);
    };
    auto load_q = [&]() {
        mbar_arrive_expect_tx(bar + 1, M::kBlocks * kTileBytes);
        for (uint32_t b = 0; b < M::kBlocks; ++b) tc::load_tile(smem + M::q + b * kTileBytes, &maps.q, 64 * b, hk, pc.row, bar + 1);
    };
    if (lead) {
        mbar_arrive_expect_tx(bar + 1, 2 * (M::kBlocks + 1) * kTileBytes);
        for (uint32_t b = 0; b < M::kBlocks; ++b) {
            tc::load_tile(smem + M::q + b * kTileBytes, &maps.q, 64 * b, hk, pc.row, bar + 1);
            tc::load_tile(smem + M::k + b * kTileBytes, &maps.k, 64 * b, hk, pc.row, bar + 1);
        }
        tc::load_tile(smem + M::v, &maps.v, 0, h, pc.row, bar + 1);
        tc::load_tile(smem + M::y, &maps.y, 0, h, pc.row, bar + 1);
    }
    // S and dS of the last tile of v, which comes first: on their way while the scores are computed
    constexpr int kStIters = DK * 8 / kTcThr;
    float sa[kStIters][8], sb[kStIters][8];
    auto fetch_states = [&](int t) {
        const int cols = min(kTile, sh.dv - t * kTile);
#pragma unroll
        for (int i = 0; i < kStIters; ++i) {
            const int at = tid + kTcThr * i, r = at >> 3, c = (at & 7) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) sa[i][j] = sb[i][j] = 0.f;
            if (r < sh.dk && c < cols) {
                const size_t o = state_at + (size_t)r * sh.dv + t * kTile + c;
                load_vec<float, 8, true>(S_in + o, sa[i]);
                load_vec<float, 8, true>(dS_out + o, sb[i]);
            }
        }
    };
    if (warp == 0) tc::alloc(s_tmem, kCols);
    TcScan my = tc_scan(g, lane, q, half == 0, s_u, s_hl, s_dec, s_tot);
    wait_for_primary();
    fetch_states(tiles - 1);
    for (int i = tid; i < 8 * kTcC; i += kTcThr) s_col[i] = 0.f;  // and s_row behind it

    unsigned phase = 0, loads = 0;
    bool ok = true;
    auto landed = [&]() {  // the loads issued are there
        ok = tc::wait(bar + 1, loads & 1) && ok;
        ++loads;
    };
    auto ready = [&]() -> bool {  // what the threads wrote is visible to the next products
        fence_proxy_async_smem();
        tc::fence_before();
        return __syncthreads_and(ok);
    };
    auto done = [&]() {  // the products issued are done
        ok = tc::wait(bar, phase & 1) && ok;
        ++phase;
        tc::fence_after();
    };
    float dot = 0.f, root = 0.f;  // e^{G_C} <dS, S>; the root of the chunk's decay
    // S and dS as fetched, split into three parts each (the third ones over Q, which is not needed between
    // the scores and dk2), and their product
    auto put_states = [&]() {
#pragma unroll
        for (int i = 0; i < kStIters; ++i) {
            const int at = tid + kTcThr * i, r = at >> 3;
            uint32_t ah[4], al[4], a3[4], bh[4], bl[4], b3[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 z = make_float2(sa[i][2 * j], sa[i][2 * j + 1]);
                const float2 a = tc::mul2(z, make_float2(root, root)), b = tc::mul2(make_float2(sb[i][2 * j], sb[i][2 * j + 1]), make_float2(root, root));
                dot = fmaf(a.x, b.x, fmaf(a.y, b.y, dot));
                ah[j] = tc::take_part(z);
                al[j] = tc::take_part(z);
                a3[j] = pack2<__nv_bfloat16>(z.x, z.y);
                z = make_float2(sb[i][2 * j], sb[i][2 * j + 1]);
                bh[j] = tc::take_part(z);
                bl[j] = tc::take_part(z);
                b3[j] = pack2<__nv_bfloat16>(z.x, z.y);
            }
            unsigned char* p = smem + M::s + tc::swz(r, at & 7);
            *reinterpret_cast<uint4*>(p) = make_uint4(ah[0], ah[1], ah[2], ah[3]);
            *reinterpret_cast<uint4*>(p + M::kS) = make_uint4(al[0], al[1], al[2], al[3]);
            *reinterpret_cast<uint4*>(p + 2 * M::kS) = make_uint4(bh[0], bh[1], bh[2], bh[3]);
            *reinterpret_cast<uint4*>(p + 3 * M::kS) = make_uint4(bl[0], bl[1], bl[2], bl[3]);
            p = smem + M::q + tc::swz(r, at & 7);
            *reinterpret_cast<uint4*>(p) = make_uint4(a3[0], a3[1], a3[2], a3[3]);
            *reinterpret_cast<uint4*>(p + M::kS) = make_uint4(b3[0], b3[1], b3[2], b3[3]);
        }
    };
    landed();
    if (n < kTcC) {  // rows of the next sequence
        tc_clear_rows(smem + M::q, M::kBlocks, n);
        tc_clear_rows(smem + M::k, M::kBlocks, n);
        tc_clear_rows(smem + M::v, 2, n);
    }
    const bool go = ready();
    tc::fence_after();
    const uint32_t tmem = *s_tmem;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
    // columns: A' and X' first; then A (bf16) 0, dv 64, dq1, dk1; last dk2, dq2 over A and dv (dk 64) or
    // over A' and X' (dk 128)
    constexpr uint32_t cA = 0, cX = 128, cAb = 0, cDv = 64;
    constexpr uint32_t cQ1 = DK == 64 ? 128 : 256, cK1 = DK == 64 ? 192 : 384, cK2 = 0, cQ2 = DK == 64 ? 64 : 128;
    const int nk = (sh.dk + 15) / 16;
    constexpr uint32_t iT = tc::idesc(128, 128, false, false);
    const uint64_t dQ = tc::desc(base + M::q, kTileBytes), dK = tc::desc(base + M::k, kTileBytes), dV = tc::desc(base + M::v, kTileBytes),
                   dY = tc::desc(base + M::y, kTileBytes), dSt = tc::desc(base + M::s, 0);  // the stride of 64-column blocks
    if (go && warp == 0) {
#pragma unroll
        for (int k = 0; k < DK / 16; ++k) {
            const uint32_t o = (k >> 2) * kTileBytes + (k & 3) * 32;
            if (k < nk) tc::mma_ss(tmem + cA, tc::ahead(dK, o), tc::ahead(dQ, o), iT, k > 0, lead);
        }
    }
    for (int t = 0; go && t < tiles; ++t) {
        if (t > 0) {
            done();
            if (lead) load_vy(t);
            landed();
            if (n < kTcC) tc_clear_rows(smem + M::v, 2, n);
            if (!ready()) break;
        }
        if (warp == 0) {
            tc::fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k) tc::mma_ss(tmem + cX, tc::ahead(dV, k * 32), tc::ahead(dY, k * 32), iT, (t | k) > 0, lead);
            tc::commit(bar, lead);
        }
    }
    float4 E = *reinterpret_cast<const float4*>(s_dec);
    const bool rises = any_rise(E);
    if (rises) {  // sums and powers of the whole chunk in place of the quarter's
        const ChunkSum s = chunk_sum(first, step, n, q);
        my.own = s.at;
        my.pow = decay_of(s.at);
        if (half == 0) {
            s_u[tok] = decay_behind(s.at, s.total);
            if (lane == 0) s_tot[2 * q] = q ? 0.f : s.total.hi, s_tot[2 * q + 1] = q ? 0.f : s.total.lo;
        }
        E = make_float4(1.f, 1.f, 1.f, 1.f);
        __syncthreads();
    }
    {
        const float2* z = reinterpret_cast<const float2*>(s_tot);
        root = root_decay_of(Exponent{(z[0].x + z[1].x) + (z[2].x + z[3].x), (z[0].y + z[1].y) + (z[2].y + z[3].y)});
    }
    const float head = sh.scale * my.pow * (q > 0 ? E.x : 1.f) * (q > 1 ? E.y : 1.f) * (q > 2 ? E.z : 1.f);
    const float tail = s_u[tok] * (q < 1 ? E.y : 1.f) * (q < 2 ? E.z : 1.f) * (q < 3 ? E.w : 1.f);
    done();
    put_states();
    // Up to 64 tokens fill half of A and P: the other half takes what bf16 leaves of them (see the forward)
    const bool brief = n <= kTcC / 2, rest = brief && half;
    const bool whole = __all_sync(0xffffffffu, ok);  // a warp takes part in what follows with all its lanes or with none
    if (rest && lane < 2) s_sum[4 * (2 + lane) + q] = 0.f;
    if (rises) {
        if (!rest && whole) weigh_pairs(lanes + cA, lanes + cX, brief ? 0 : 2 * half, q, my.own, first, step, n, sh.scale, s_row, s_col, s_sum);
        my.diag = 1.f;
        __syncthreads();
        if (half == 0) s_u[tok] = s_hl[tok] = 1.f;
        tc::fence_before();
        __syncthreads();
        tc::fence_after();
    }
    uint32_t ab[2][16], pb[2][16];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int grp = (brief ? 0 : 2 * half) + e;  // 32 columns i
        if (grp < q || !whole) {
#pragma unroll
            for (int j = 0; j < 16; ++j) ab[e][j] = pb[e][j] = 0u;
            continue;
        }
        float m[32];
        // row factor: this j's weight up to the group's first token, or exp2(-L_j) inside its quarter
        const float f = sh.scale * (grp == q ? my.diag : s_u[tok] * (q < 1 && grp > 1 ? E.y : 1.f) * (q < 2 && grp > 2 ? E.z : 1.f));
        const float2 f2 = make_float2(f, f);
        const bool pairs = grp == q && my.diag < 0.f;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float a[16], b[16];
            tc::ld16(lanes + cA + 32 * grp + 16 * s, a);
            tc::ld16(lanes + cX + 32 * grp + 16 * s, b);
            tc::wait_ld();
            if (!pairs && !rest) {
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 z = *reinterpret_cast<const float4*>(s_hl + 32 * grp + 16 * s + j);
#pragma unroll
                    for (int e2 = 0; e2 < 4; e2 += 2) {
                        const float2 w = tc::mul2(f2, e2 ? make_float2(z.z, z.w) : make_float2(z.x, z.y));
                        const float2 x2 = make_float2(b[j + e2], b[j + e2 + 1]);
                        const float2 aw = tc::mul2(make_float2(a[j + e2], a[j + e2 + 1]), w), bw = tc::mul2(x2, w), mw = tc::mul2(aw, x2);
                        ab[e][8 * s + (j + e2) / 2] = pack2<__nv_bfloat16>(aw.x, aw.y);
                        pb[e][8 * s + (j + e2) / 2] = pack2<__nv_bfloat16>(bw.x, bw.y);
                        m[16 * s + j + e2] = mw.x;
                        m[16 * s + j + e2 + 1] = mw.y;
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    Exponent o;
                    o.hi = __shfl_sync(0xffffffffu, my.own.hi, 16 * s + j);
                    o.lo = __shfl_sync(0xffffffffu, my.own.lo, 16 * s + j);
                    const float w = pairs ? sh.scale * decay_between(o, my.own) : f * s_hl[32 * grp + 16 * s + j], aw = a[j] * w;
                    m[16 * s + j] = aw * b[j];
                    a[j] = aw;
                    b[j] *= w;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float2 x2 = make_float2(a[2 * j], a[2 * j + 1]), y2 = make_float2(b[2 * j], b[2 * j + 1]);
                    ab[e][8 * s + j] = tc::take_part(x2);
                    pb[e][8 * s + j] = tc::take_part(y2);
                    if (rest) {
                        ab[e][8 * s + j] = pack2<__nv_bfloat16>(x2.x, x2.y);
                        pb[e][8 * s + j] = pack2<__nv_bfloat16>(y2.x, y2.y);
                    }
                }
            }
        }
        if (grp == q) {  // before the pair's earlier token there is no weight, whatever the score
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const uint32_t in = lane < 2 * j + 1 ? (lane <= 2 * j ? 0xffffffffu : 0u) : lane == 2 * j + 1 ? 0xffff0000u : 0u;
                ab[e][j] &= in;
                pb[e][j] &= in;
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) m[j] = j >= lane ? m[j] : 0.f;
        }
        if (rest || rises) continue;
        pair_sums(m, grp, q, lane, s_row, s_col, s_sum);
    }
    // A over the scores (all warps of the quarter have read them)
    tc::fence_before();
    asm volatile("bar.sync %0, 64;" : : "r"(1 + q) : "memory");
    tc::fence_after();
    tc::st16(lanes + cAb + 32 * half, ab[0]);
    tc::st16(lanes + cAb + 32 * half + 16, ab[1]);
    tc::wait_st();

    constexpr uint32_t iV = tc::idesc(128, 64, false, true);   // B: rows K, columns N
    constexpr uint32_t iK = tc::idesc(128, DK, false, false);  // B: rows N, columns K
    const bool wide_v = sh.dv % 16 == 0 && ((uintptr_t)out.dv & 31u) == 0;
    for (int t = tiles - 1; t >= 0; --t) {
        if (t != tiles - 1) {
            landed();
            if (n < kTcC) tc_clear_rows(smem + M::v, 2, n);
        }
        if (!ready()) break;
        if (warp == 0) {
            tc::fence_after();
            const bool first = t == tiles - 1;
#pragma unroll
            for (int k = 0; k < DK / 16; ++k)
                if (k < nk) {
                    const uint64_t a = tc::ahead(dK, (k >> 2) * kTileBytes + (k & 3) * 32);
                    tc::mma_ss(tmem + cDv, a, tc::ahead(dSt, 2 * M::kS + k * 2048), iV, k > 0, lead);
                    tc::mma_ss(tmem + cDv, a, tc::ahead(dSt, 3 * M::kS + k * 2048), iV, 1, lead);
                }
            // one accumulator after the other: switching between them costs more than a product; small parts first
#pragma unroll
            for (int i = 2; i >= 0; --i)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc::mma_ss(tmem + cQ1, tc::ahead(dY, k * 32), tc::ahead(i < 2 ? dSt : dQ, (i < 2 ? i * M::kS : 0) + k * 32), iK,
                               i < 2 || k > 0 || !first, lead);
#pragma unroll
            for (int i = 2; i >= 0; --i)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc::mma_ss(tmem + cK1, tc::ahead(dV, k * 32), tc::ahead(i < 2 ? dSt : dQ, (i < 2 ? 2 + i : 1) * M::kS + k * 32), iK,
                               i < 2 || k > 0 || !first, lead);
            tc::commit(bar, lead);
        }
        done();
        float dv[32];
        tc::ld32(lanes + cDv + 32 * half, dv);
        tc::wait_ld();
        tc::fence_before();
        if (!__syncthreads_and(ok)) break;
        if (warp == 0) {
            tc::fence_after();
#pragma unroll
            for (int k = 0; k < kTcC / 16; ++k)
                tc::mma_ts(tmem + cDv, tmem + cAb + 8 * k, tc::ahead(dY, (k & (brief ? 3 : 7)) * 2048), iV, k > 0, lead);
            tc::commit(bar, lead);
        }
        if (t > 0) {
            fetch_states(t - 1);
            put_states();
        }
        done();
        if (lead) {
            if (t > 0) load_vy(t - 1);
            else load_q();
        }
        const int cols = min(kTile, sh.dv - t * kTile);
        __nv_bfloat16* o = (__nv_bfloat16*)out.dv + ((size_t)(pc.row + tok) * sh.H + h) * sh.dv + t * kTile + 32 * half;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float b[16];
            tc::ld16(lanes + cDv + 32 * half + 16 * j, b);
            tc::wait_ld();
            uint32_t r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                r[i] = pack2<__nv_bfloat16>(fmaf(tail, dv[16 * j + 2 * i], b[2 * i]), fmaf(tail, dv[16 * j + 2 * i + 1], b[2 * i + 1]));
            if (ok && tok < n) store_row16(o + 16 * j, r, 32 * half + 16 * j, cols, wide_v);
        }
    }
    // P over V and dY: rows j, two blocks of 64 columns i
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(smem + M::v + half * kTileBytes + tc::swz(tok, 4 * e + c)) =
                make_uint4(pb[e][4 * c], pb[e][4 * c + 1], pb[e][4 * c + 2], pb[e][4 * c + 3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) s_red[warp] = dot;
    landed();
    if (n < kTcC) tc_clear_rows(smem + M::q, M::kBlocks, n);
    if (ready()) {
        if (warp == 0) {
            tc::fence_after();
            constexpr uint32_t iK2 = tc::idesc(128, DK, false, true), iQ2 = tc::idesc(128, DK, true, true);
#pragma unroll
            for (int k = 0; k < kTcC / 16; ++k)
                tc::mma_ss(tmem + cK2, tc::ahead(dV, (k >> 2) * kTileBytes + (k & 3) * 32), tc::ahead(dQ, (k & (brief ? 3 : 7)) * 2048), iK2,
                           k > 0, lead);
            // of a short chunk the two parts' columns, one tile after the other, over the same rows j; rows of the
            // product behind the 64th, into which the second tile or what lies behind it goes, are no tokens
#pragma unroll
            for (int k = 0; k < kTcC / 16; ++k)
                tc::mma_ss(tmem + cQ2, tc::ahead(dV, brief ? (k >> 2) * kTileBytes + (k & 3) * 2048 : k * 2048),
                           tc::ahead(dK, (k & (brief ? 3 : 7)) * 2048), iQ2, k > 0, lead);
            tc::commit(bar, lead);
        }
        done();
        // this thread's row of dq and dk: half of the channels, 16 at a time
        constexpr int kHalf = DK / 2;
        const bool wide_k = sh.dk % 16 == 0 && (((uintptr_t)out.dq | (uintptr_t)out.dk) & 31u) == 0;
        float iq = 0.f, ok_ = 0.f;
#pragma unroll 1
        for (int c = half * kHalf; c < (half + 1) * kHalf; c += 16) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {  // dq, dk
                float a[16], b[16];
                tc::ld16(lanes + (w ? cK1 : cQ1) + c, a);
                tc::ld16(lanes + (w ? cK2 : cQ2) + c, b);
                tc::wait_ld();
                const float f = w ? tail : head;
                float in = 0.f;
                const unsigned char* tile = smem + (w ? M::k : M::q) + (c >> 6) * kTileBytes;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 v = *reinterpret_cast<const uint4*>(tile + tc::swz(tok, ((c & 63) >> 3) + j));
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 z = unpack2<__nv_bfloat16>(u[i]);
                        a[8 * j + 2 * i] *= f;
                        a[8 * j + 2 * i + 1] *= f;
                        in = fmaf(a[8 * j + 2 * i], z.x, fmaf(a[8 * j + 2 * i + 1], z.y, in));
                    }
                }
                if (w) ok_ += in;
                else iq += in;
#pragma unroll
                for (int j = 0; j < 16; ++j) a[j] += b[j];
                if (ok && tok < n) {
                    if (out.partial) {
                        float* o = (float*)(w ? out.dk : out.dq) + ((size_t)(pc.row + tok) * sh.H + h) * sh.dk + c;
#pragma unroll
                        for (int j = 0; j < 16; j += 8)
                            if (c + j < sh.dk) {  // dk is a multiple of 8
                                uint32_t r[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(a[j + i]);
                                store_32(o + j, r);
                            }
                    } else {
                        __nv_bfloat16* o = (__nv_bfloat16*)(w ? out.dk : out.dq) + ((size_t)(pc.row + tok) * sh.Hk + hk) * sh.dk + c;
                        uint32_t r[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) r[j] = pack2<__nv_bfloat16>(a[2 * j], a[2 * j + 1]);
                        store_row16(o, r, c, sh.dk, wide_k);
                    }
                }
            }
        }
        s_in[half * kTcC + tok] = iq;
        s_out[half * kTcC + tok] = ok_;
        iq = warp_total(iq);
        ok_ = warp_total(ok_);
        if (lane == 0) {
            s_sum[16 + 4 * half + q] = iq;
            s_sum[24 + 4 * half + q] = ok_;
        }
    }
    if (!ok) set_status(status, kStatusTimeout);
    tc::fence_before();
    __syncthreads();
    if (warp == 0) tc::dealloc(tmem, kCols);
    // dg of token t = tok (warps 0 .. 3)
    if (half == 0) {
        float d = 0.f;
        for (int i = 0; i <= q; ++i) d += s_col[i * kTcC + tok];
        // rows j < t: their pairs in later groups of columns, and what leaves through the state; rows i >= t:
        // what enters through the state.  Other quarters by their sums, this one's by a scan.
        float left = s_out[tok] + s_out[kTcC + tok], right = s_in[tok] + s_in[kTcC + tok];
        for (int gr = q + 1; gr < 4; ++gr) {
            left += s_row[gr * kTcC + tok];
            d += s_sum[16 + gr] + s_sum[20 + gr];
        }
        for (int m = 0; m < q; ++m) {
            d += s_sum[24 + m] + s_sum[28 + m];
            for (int gr = q + 1; gr < 4; ++gr) d += s_sum[4 * gr + m];
        }
        float pre = __shfl_up_sync(0xffffffffu, left, 1), suf = right;  // tokens before this one; from this one on
        if (lane == 0) pre = 0.f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, pre, o), z = __shfl_down_sync(0xffffffffu, suf, o);
            if (lane >= o) pre += y;
            if (lane + o < 32) suf += z;
        }
        d += pre + suf;
        float z = 0.f;
        for (int i = 0; i < 8; ++i) z += s_red[i];
        d += z;
        if (tok >= n) d = 0.f;
        if (!sh.head_decay) {
            if (ok && tok < n) out.dg[(size_t)(pc.row + tok) * sh.H + h] = d;
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
            if (lane == 0) s_u[q] = d;
        }
    }
    if (sh.head_decay) {
        __syncthreads();
        if (tid == 0 && ok) out.dg[(size_t)id * sh.H + h] = (s_u[0] + s_u[1]) + (s_u[2] + s_u[3]);
    }
}

}  // namespace la
}  // namespace fv
