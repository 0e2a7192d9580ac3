// kda_latent_bwd.hip -- the gradient of latent attention in its expanded form
// (kda_latent_bwd in include/kda_latent.h).
//
// Two passes over the pairs of queries and keys, each with the sums that it can keep
// in accumulators, so that nothing is added up in memory in an order left to chance:
//   dq:  a workgroup has 128 queries and runs through the keys they see,
//        S^T = K Q^T, dP^T = V dO^T, dQ^T += K^T dS^T          (32 products a 32 x 32 block)
//   dkv: a workgroup has 128 keys and runs through the queries that see them,
//        S = Q K^T, dP = dO V^T, dV^T += dO^T P, dK^T += Q^T dS   (40 products)
// with P = e^(scale S - lse) and dS = P (dP - delta).  (One pass would take S and dP
// once, 52 products instead of 72, but add dQ up in fp32 memory.)  As in the forward a
// wave has 32 of its own side's tokens in registers, the lane's column, and the other side's come
// through LDS, 64 at a time; P and dS are fed back as B operands as they stand.  A unit is
// 32 tokens of the other side: the first products of unit u + 1 run beside the
// exponentials of unit u.  Every head leaves its part of dk_pe in fp32; they are added up
// in the order of the heads.  Few blocks take one launch for both passes, and parts of their
// other side each, which are added up in their order by a launch of its own.
//
// The matrix instructions bound it, with one wave a SIMD, whose 512 registers hold its sums:
// 8192 tokens x 32 heads take 982 to 1022 us for dq (1.12 to 1.08 PFLOP/s), 1212 to 1241 for
// dkv (1.13 to 1.11) and 12 for dk_pe; a large matrix product reaches 1.2 to 1.36.
//
// Precision: fp32 but for P and dS, rounded to bf16 for the products they enter (at most 2^-8 of
// each, as large as the outputs' own rounding); delta and lse are fp32.
#include "kda_latent_common.h"

namespace kda {

namespace {

constexpr int kBlock = kLatentBwdBlock;

// P and dS of unit entries: x in 0 .. 15 a probability, then 16 .. 31 a dS.
struct Pairs {
    uint32_t p[8], e[8];
    float last;
};
__device__ __forceinline__ s8 operand_of(const uint32_t (&w)[8], int s) {
    const u4v v = {w[4 * s], w[4 * s + 1], w[4 * s + 2], w[4 * s + 3]};
    return __builtin_bit_cast(s8, v);
}

// S and dP go to ordinary registers, where the vector instructions take them, while the
// sums over all pairs stay in the accumulator half of the file: the compiler, which uses
// one half for all products of a kernel, would move 128 values a tile.  What it does not
// see is that results are there some 11 issue slots after the last product only: between a
// unit's first products and their first use lie the 12 or 20 products of its sums, or
// products_done.
__device__ __forceinline__ void first_product(f16v &d, const s8 &a, const s8 &b) {
    asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, 0" : "=&v"(d) : "v"(a), "v"(b));
}
__device__ __forceinline__ void add_product(f16v &d, const s8 &a, const s8 &b) {
    asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(d) : "v"(a), "v"(b));
}
__device__ __forceinline__ void products_done() { asm volatile("s_nop 15\n\ts_nop 7" ::: "memory"); }

// ---- dq -----------------------------------------------------------------------------

constexpr int kStages = 3;  // tiles in LDS: two in use, one on its way
struct DqSmem {
    uint16_t kn[kStages][kKeys * kNope];
    uint16_t kp[kStages][kKeys * kPe];
    uint16_t v[kStages][kKeys * kVal];
};
struct DqState {
    s8 q[kQk / 16], y[kVal / 16];
    f16v dq[kQk / 32];
    float lse2, delta;
};
struct DqAddr {
    uint32_t kn, kp, v;      // row operands in buffer 0
    uint32_t tn, tp;         // column operands
};

// Slots of a unit: the first products of the next one, S and dP in turn, then dQ's.
constexpr int kSdSlots = kQk / 16 + kVal / 16;
__device__ __forceinline__ bool is_s(int n) { return n < 2 * kVal / 16 ? (n & 1) == 0 : true; }
__device__ __forceinline__ int sd_block(int n) { return n < 2 * kVal / 16 ? n >> 1 : n - kVal / 16; }

template <bool NEXT>
__device__ __forceinline__ void dq_unit(DqState &f, const DqAddr &at, int buf, int half, int nbuf, int nhalf, f16v &s, f16v &dp,
                                        f16v &s2, f16v &dp2, float c) {
    constexpr int kAhead = 4, kFirst = NEXT ? 0 : kSdSlots, kAll = kSdSlots + 2 * kQk / 32;
    Pairs w;
    const auto operand = [&](int n) -> s8 {
        if (n < kSdSlots) {
            const int ks = sd_block(n);
            if (!is_s(n)) return row_operand<2 * kVal>(at.v + nbuf * (uint32_t)sizeof(DqSmem::v[0]), nhalf, ks);
            return ks < kNope / 16 ? row_operand<2 * kNope>(at.kn + nbuf * (uint32_t)sizeof(DqSmem::kn[0]), nhalf, ks)
                                   : row_operand<2 * kPe>(at.kp + nbuf * (uint32_t)sizeof(DqSmem::kp[0]), nhalf, ks - kNope / 16);
        }
        const int m = n - kSdSlots, ks = m / (kQk / 32), dt = m % (kQk / 32);
        return dt < kNope / 32 ? col_operand<2 * kNope>(at.tn + buf * (uint32_t)sizeof(DqSmem::kn[0]), 2 * half + ks, dt)
                               : col_operand<2 * kPe>(at.tp + buf * (uint32_t)sizeof(DqSmem::kp[0]), 2 * half + ks, dt - kNope / 32);
    };
    const auto pair = [&](int i) {  // dS of entry i
        const float e = __builtin_amdgcn_exp2f(fmaf(s[i], c, -f.lse2)) * (dp[i] - f.delta);
        if (i & 1) w.e[i / 2] = pack2(w.last, e);
        else w.last = e;
    };
    s8 ring[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) ring[(kFirst + n) % kAhead] = operand(kFirst + n);
    if (!NEXT) {
#pragma unroll
        for (int i = 0; i < 16; ++i) pair(i);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = kFirst; n < kAll; ++n) {
        const s8 a = ring[n % kAhead];
        const int m = n - kSdSlots;
        if (m >= 0) f.dq[m % (kQk / 32)] = mfma32(a, operand_of(w.e, m / (kQk / 32)), f.dq[m % (kQk / 32)]);
        else if (n == 0) first_product(s2, a, f.q[0]);
        else if (n == 1) first_product(dp2, a, f.y[0]);
        else if (is_s(n)) add_product(s2, a, f.q[sd_block(n)]);
        else add_product(dp2, a, f.y[sd_block(n)]);
        if (n + kAhead < kAll) ring[n % kAhead] = operand(n + kAhead);
        if (NEXT && n < 16) pair(n);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// A row's lse in log2 units (0 where no key is seen) and d_out . out.  The lanes n and n + 32 have a row,
// 8 values of every 16 each (y: d_out's); both get the results.
struct Stat {
    float lse2, delta;
};
__device__ __forceinline__ Stat row_stat(const s8 (&y)[kVal / 16], const uint16_t *o, float lse) {
    float d = 0.0f;
#pragma unroll
    for (int ks = 0; ks < kVal / 16; ++ks) {
        const s8 v = *reinterpret_cast<const s8 *>(o + 16 * ks);
#pragma unroll
        for (int j = 0; j < 8; ++j) d = fmaf(bf16_bits_to_f32((uint16_t)y[ks][j]), bf16_bits_to_f32((uint16_t)v[j]), d);
    }
    return {lse == -INFINITY ? 0.0f : lse * kLog2e, pair_sum(d)};
}

// What a workgroup leaves of its part of a block: GROUPS groups of 32 values of a wave's 32 tokens, an
// accumulator each.
template <int GROUPS>
__device__ __forceinline__ f4 *part_of(const LatentArgs &a, int64_t place, int wave, int group) {
    return reinterpret_cast<f4 *>(a.part) + ((place * 4 + wave) * GROUPS + group) * 4 * 64 + (threadIdx.x & 63);
}
__device__ __forceinline__ void leave(f4 *p, const f16v &v, float scale) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
        p[e * 64] = f4{v[4 * e] * scale, v[4 * e + 1] * scale, v[4 * e + 2] * scale, v[4 * e + 3] * scale};
}

// place: the block, counted over the heads, with SPLIT its part.  STORE: the rows' statistics too, for dkv.
template <bool STORE, bool SPLIT>
__device__ __forceinline__ void dq_block(const LatentArgs &a, int64_t place, DqSmem &sm) {
    const int64_t unit = SPLIT ? place / a.parts : place;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t h = unit % a.H;
    Span sp;
    if (!span_of<kBlock, false>(a, unit / a.H, a.causal, sp)) return;
    const int q_first = sp.block * kBlock + wave * 32;
    const int block_last = min(sp.lq, (sp.block + 1) * kBlock) - 1;
    if (block_last < sp.block * kBlock) return;
    const auto sees = [&](int i) { return a.causal ? max(0, min(sp.lk, i + 1 + sp.lk - sp.lq)) : sp.lk; };
    const int all = (sees(block_last) + kKeys - 1) / kKeys;
    const int part_tiles = SPLIT ? part_tiles_of(a, (sp.lk + kKeys - 1) / kKeys) : 0;
    const int t0 = SPLIT ? (int)(place - unit * a.parts) * part_tiles : 0;
    if (SPLIT && t0 >= max(all, 1)) return;
    const int tiles = SPLIT ? min(all, t0 + part_tiles) : all;
    const int last = min(sp.lq - 1, q_first + 31);
    const int mine = last < q_first ? 0 : min(tiles, (sees(last) + kKeys - 1) / kKeys);  // of this wave
    const int whole = sees(q_first) / 32;                                    // units without hidden keys

    const uint16_t *kv = a.kv + sp.b * a.kvb + sp.k0 * a.kvt + h * kKvRow;
    const uint16_t *pe = a.pe + sp.b * a.peb + sp.k0 * a.pet;
    const uint32_t kv_bytes = (uint32_t)a.kvt * 2, pe_bytes = (uint32_t)a.pet * 2;
    const uint32_t off_n = tile_offset<kNope>(tid, kv_bytes), off_p = tile_offset<kPe>(tid, pe_bytes);
    const uint32_t lds_kn = lds_addr(sm.kn), lds_kp = lds_addr(sm.kp), lds_v = lds_addr(sm.v);
    const auto copy = [&](int j) {
        if (j >= tiles) return;
        const int rows = min(kKeys, sp.lk - j * kKeys), buf = j % kStages;
        const uint16_t *p = kv + (int64_t)j * kKeys * a.kvt;
        copy_tile<kNope>(p, rows, kv_bytes, off_n, lds_kn + buf * (uint32_t)sizeof(sm.kn[0]), wave);
        copy_tile<kPe>(pe + (int64_t)j * kKeys * a.pet, rows, pe_bytes, off_p, lds_kp + buf * (uint32_t)sizeof(sm.kp[0]), wave);
        copy_tile<kVal>(p + kNope, rows, kv_bytes, off_n, lds_v + buf * (uint32_t)sizeof(sm.v[0]), wave);
    };
    copy(t0);
    copy(t0 + 1);

    DqState f;
    const int i = q_first + (lane & 31), row = min(i, sp.lq - 1);  // rows behind the last: of no effect, not stored
    const int seen = sees(i);
    {
        const int64_t t = sp.b * a.T + sp.q0 + row;
        const uint16_t *q = a.q + sp.b * a.qb + (sp.q0 + row) * a.qt + h * kQk + 8 * g;
        const uint16_t *y = a.dy + sp.b * a.yb + (sp.q0 + row) * a.yt + h * kVal + 8 * g;
        const uint16_t *o = a.o + sp.b * a.ob + (sp.q0 + row) * a.ot + h * kVal + 8 * g;
#pragma unroll
        for (int ks = 0; ks < kQk / 16; ++ks) f.q[ks] = *reinterpret_cast<const s8 *>(q + 16 * ks);
#pragma unroll
        for (int ks = 0; ks < kVal / 16; ++ks) f.y[ks] = *reinterpret_cast<const s8 *>(y + 16 * ks);
        const Stat st = row_stat(f.y, o, a.lse_in[t * a.H + h]);
        f.lse2 = st.lse2;
        f.delta = st.delta;
        if (STORE && g == 0 && i < sp.lq) {
            float *stat = a.stat + h * a.B * a.T + t;
            stat[0] = st.lse2;
            stat[a.H * a.B * a.T] = st.delta;
        }
    }
#pragma unroll
    for (int d = 0; d < kQk / 32; ++d) f.dq[d] = zero16();
    const DqAddr at = {row_at<2 * kNope>(lds_kn, lane), row_at<2 * kPe>(lds_kp, lane), row_at<2 * kVal>(lds_v, lane),
                       col_at<2 * kNope>(lds_kn, lane), col_at<2 * kPe>(lds_kp, lane)};
    const float c = a.scale * kLog2e;

    const auto hide = [&](int u, f16v &s) {
        if (u < whole) return;
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = u * 32 + 8 * (e / 4) + 4 * g + e % 4 < seen ? s[e] : -INFINITY;
    };
    // Tile t is there and tile t - 1 read, whose place the next copies take.
    const auto begin = [&](int t) {
        copies_done();
        copy(t + 1);
    };
    int t = t0;
    if (tiles > t0) copies_done();
    if (mine > t0) {
        f16v s0, d0, s1, d1;
        int st = t0 % kStages;
#pragma unroll
        for (int n = 0; n < kSdSlots; ++n) {
            const int ks = sd_block(n);
            if (is_s(n)) {
                const uint32_t kn = at.kn + st * (uint32_t)sizeof(sm.kn[0]), kp = at.kp + st * (uint32_t)sizeof(sm.kp[0]);
                const s8 x = ks < kNope / 16 ? row_operand<2 * kNope>(kn, 0, ks) : row_operand<2 * kPe>(kp, 0, ks - kNope / 16);
                if (n == 0) first_product(s0, x, f.q[ks]);
                else add_product(s0, x, f.q[ks]);
            } else {
                const s8 x = row_operand<2 * kVal>(at.v + st * (uint32_t)sizeof(sm.v[0]), 0, ks);
                if (n == 1) first_product(d0, x, f.y[ks]);
                else add_product(d0, x, f.y[ks]);
            }
            if (n % 4 == 3) __builtin_amdgcn_sched_barrier(0);
        }
        products_done();
        for (; t < mine - 1; ++t) {
            const int next = st == kStages - 1 ? 0 : st + 1;
            begin(t + 1);
            hide(2 * t, s0);
            dq_unit<true>(f, at, st, 0, st, 1, s0, d0, s1, d1, c);
            hide(2 * t + 1, s1);
            dq_unit<true>(f, at, st, 1, next, 0, s1, d1, s0, d0, c);
            st = next;
        }
        hide(2 * t, s0);
        dq_unit<true>(f, at, st, 0, st, 1, s0, d0, s1, d1, c);
        hide(2 * t + 1, s1);
        dq_unit<false>(f, at, st, 1, 0, 0, s1, d1, s0, d0, c);
        ++t;
    } else {
        ++t;
    }
    for (; t < tiles; ++t) begin(t);

    if (SPLIT && all > part_tiles) {
#pragma unroll
        for (int d = 0; d < kQk / 32; ++d) leave(part_of<kQk / 32>(a, place, wave, d), f.dq[d], a.scale);
        return;
    }
    __syncthreads();  // the tiles are read
    char *stage = reinterpret_cast<char *>(&sm) + wave * 32 * 2 * kQk;
    static_assert(sizeof(sm) >= 4 * 32 * 2 * kQk, "");
#pragma unroll
    for (int d = 0; d < kQk / 32; ++d) stage_values<kQk / 8>(stage, lane, 4 * d, f.dq[d], a.scale);
    store_rows<kQk / 8>(stage, lane, a.dq + ((sp.b * a.T + sp.q0 + q_first) * a.H + h) * kQk, a.H * kQk, sp.lq - q_first);
}

__global__ __launch_bounds__(256, 1) void latent_dq_kernel(LatentArgs a) {
    __shared__ __attribute__((aligned(1024))) DqSmem sm;
    dq_block<true, false>(a, a.base + blockIdx.x, sm);
}

// ---- dkv ----------------------------------------------------------------------------

struct DkvSmem {
    uint16_t qn[kStages][kKeys * kNope];
    uint16_t qp[kStages][kKeys * kPe];
    uint16_t y[kStages][kKeys * kVal];
    float lse2[kStages][kKeys], delta[kStages][kKeys];
};
struct DkvState {
    s8 k[kQk / 16], v[kVal / 16];
    f16v dk[kQk / 32], dv[kVal / 32];
};
struct DkvAddr {
    uint32_t qn, qp, y;      // row operands in stage 0
    uint32_t tn, tp, ty;     // column operands
    uint32_t stat;           // lse2 of the lane's first query
};
typedef const __attribute__((address_space(3))) f4 *lds_f4;

template <bool NEXT>
__device__ __forceinline__ void dkv_unit(DkvState &f, const DkvAddr &at, int st, int half, int nst, int nhalf, f16v &s, f16v &dp,
                                         f16v &s2, f16v &dp2, float c) {
    constexpr int kAhead = 4, kFirst = NEXT ? 0 : kSdSlots, kDv = 2 * kVal / 32, kAll = kSdSlots + kDv + 2 * kQk / 32;
    Pairs w;
    f4 lse2[4], delta[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t p = at.stat + st * (kKeys * 4) + half * 128 + e * 32;
        lse2[e] = *reinterpret_cast<lds_f4>(p);
        delta[e] = *reinterpret_cast<lds_f4>(p + (uint32_t)sizeof(DkvSmem::lse2));
    }
    const auto operand = [&](int n) -> s8 {
        if (n < kSdSlots) {
            const int ks = sd_block(n);
            if (!is_s(n)) return row_operand<2 * kVal>(at.y + nst * (uint32_t)sizeof(DkvSmem::y[0]), nhalf, ks);
            return ks < kNope / 16 ? row_operand<2 * kNope>(at.qn + nst * (uint32_t)sizeof(DkvSmem::qn[0]), nhalf, ks)
                                   : row_operand<2 * kPe>(at.qp + nst * (uint32_t)sizeof(DkvSmem::qp[0]), nhalf, ks - kNope / 16);
        }
        int m = n - kSdSlots;
        if (m < kDv) return col_operand<2 * kVal>(at.ty + st * (uint32_t)sizeof(DkvSmem::y[0]), 2 * half + m / (kVal / 32), m % (kVal / 32));
        m -= kDv;
        const int ks = 2 * half + m / (kQk / 32), dt = m % (kQk / 32);
        return dt < kNope / 32 ? col_operand<2 * kNope>(at.tn + st * (uint32_t)sizeof(DkvSmem::qn[0]), ks, dt)
                               : col_operand<2 * kPe>(at.tp + st * (uint32_t)sizeof(DkvSmem::qp[0]), ks, dt - kNope / 32);
    };
    // Entry i's probability takes the place of its score.
    const auto prob = [&](int i) {
        s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -lse2[i / 4][i % 4]));
        if (i & 1) w.p[i / 2] = pack2(s[i - 1], s[i]);
    };
    const auto pair = [&](int i) {
        const float e = s[i] * (dp[i] - delta[i / 4][i % 4]);
        if (i & 1) w.e[i / 2] = pack2(w.last, e);
        else w.last = e;
    };
    s8 ring[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) ring[(kFirst + n) % kAhead] = operand(kFirst + n);
    if (!NEXT) {
#pragma unroll
        for (int i = 0; i < 16; ++i) prob(i);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = kFirst; n < kAll; ++n) {
        const s8 a = ring[n % kAhead];
        const int m = n - kSdSlots;
        if (m >= kDv) {
            const int x = m - kDv;
            f.dk[x % (kQk / 32)] = mfma32(a, operand_of(w.e, x / (kQk / 32)), f.dk[x % (kQk / 32)]);
        } else if (m >= 0) {
            f.dv[m % (kVal / 32)] = mfma32(a, operand_of(w.p, m / (kVal / 32)), f.dv[m % (kVal / 32)]);
        } else if (n < 2) {
            if (n == 0) first_product(s2, a, f.k[0]);
            else first_product(dp2, a, f.v[0]);
        } else if (is_s(n)) {
            add_product(s2, a, f.k[sd_block(n)]);
        } else {
            add_product(dp2, a, f.v[sd_block(n)]);
        }
        if (n + kAhead < kAll) ring[n % kAhead] = operand(n + kAhead);
        if (NEXT && n < 16) prob(n);
        if (m >= 0 && m < kDv) {  // dS, which the products behind these take
            pair(2 * m);
            pair(2 * m + 1);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

constexpr int kDkvGroups = (kQk + kVal) / 32;
template <bool SPLIT>
__device__ __forceinline__ void dkv_block(const LatentArgs &a, int64_t place, DkvSmem &sm) {
    const int64_t unit = SPLIT ? place / a.parts : place;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t h = unit % a.H;
    Span sp;
    if (!span_of<kBlock, true>(a, unit / a.H, false, sp)) return;
    if (sp.block * kBlock >= sp.lk) return;
    const int k_first = sp.block * kBlock + wave * 32;
    // The first query that sees key j, and with it all behind it.
    const int lead = sp.lk - sp.lq;
    const auto seen_from = [&](int j) { return a.causal ? max(0, j - lead) : 0; };
    const int first_all = seen_from(sp.block * kBlock) / kKeys;                // tiles of queries
    const int tiles_all = max(first_all, (sp.lq + kKeys - 1) / kKeys);         // (one behind the last)
    const int part_tiles = SPLIT ? part_tiles_of(a, (sp.lq + kKeys - 1) / kKeys) : 0;
    const int first = SPLIT ? first_all + (int)(place - unit * a.parts) * part_tiles : first_all;
    if (SPLIT && first > first_all && first >= tiles_all) return;
    const int tiles = SPLIT ? min(tiles_all, first + part_tiles) : tiles_all;
    const int j = k_first + (lane & 31), row = min(j, sp.lk - 1);
    const int from = seen_from(j);                                    // of the lane's key
    const int top_key = min(k_first + 31, sp.lk - 1);
    const int whole = (seen_from(top_key) + 31) / 32;                 // units from here on see all of the wave's keys
    const int full = sp.lq / 32;                                      // units behind these are not full

    const int64_t tok = sp.b * a.T + sp.q0;
    const uint16_t *q = a.q + sp.b * a.qb + sp.q0 * a.qt + h * kQk;
    const uint16_t *y = a.dy + sp.b * a.yb + sp.q0 * a.yt + h * kVal;
    const float *stat = a.stat + h * a.B * a.T + tok;
    const uint32_t q_bytes = (uint32_t)a.qt * 2, y_bytes = (uint32_t)a.yt * 2;
    const uint32_t off_n = tile_offset<kNope>(tid, q_bytes), off_p = tile_offset<kPe>(tid, q_bytes),
                   off_y = tile_offset<kVal>(tid, y_bytes);
    const uint32_t lds_qn = lds_addr(sm.qn), lds_qp = lds_addr(sm.qp), lds_y = lds_addr(sm.y), lds_l = lds_addr(sm.lse2),
                   lds_d = lds_addr(sm.delta);
    const auto copy = [&](int t) {
        if (t >= tiles) return;
        const int rows = min(kKeys, sp.lq - t * kKeys), st = t % kStages;
        const uint16_t *p = q + (int64_t)t * kKeys * a.qt;
        copy_tile<kNope>(p, rows, q_bytes, off_n, lds_qn + st * (uint32_t)sizeof(sm.qn[0]), wave);
        copy_tile<kPe>(p + kNope, rows, q_bytes, off_p, lds_qp + st * (uint32_t)sizeof(sm.qp[0]), wave);
        copy_tile<kVal>(y + (int64_t)t * kKeys * a.yt, rows, y_bytes, off_y, lds_y + st * (uint32_t)sizeof(sm.y[0]), wave);
        if (wave < 2) {
            const float *x = stat + (wave ? a.H * a.B * a.T : 0) + (int64_t)t * kKeys;
            copy4(buffer_of(x, (uint32_t)rows * 4), (uint32_t)lane * 4, (wave ? lds_d : lds_l) + st * (kKeys * 4));
        }
    };
    copy(first);
    copy(first + 1);

    DkvState f;
    {
        const uint16_t *kv = a.kv + sp.b * a.kvb + (sp.k0 + row) * a.kvt + h * kKvRow + 8 * g;
        const uint16_t *pe = a.pe + sp.b * a.peb + (sp.k0 + row) * a.pet + 8 * g;
#pragma unroll
        for (int ks = 0; ks < kQk / 16; ++ks)
            f.k[ks] = ks < kNope / 16 ? *reinterpret_cast<const s8 *>(kv + 16 * ks)
                                      : *reinterpret_cast<const s8 *>(pe + 16 * ks - kNope);
#pragma unroll
        for (int ks = 0; ks < kVal / 16; ++ks) f.v[ks] = *reinterpret_cast<const s8 *>(kv + kNope + 16 * ks);
    }
#pragma unroll
    for (int d = 0; d < kQk / 32; ++d) f.dk[d] = zero16();
#pragma unroll
    for (int d = 0; d < kVal / 32; ++d) f.dv[d] = zero16();
    const DkvAddr at = {row_at<2 * kNope>(lds_qn, lane), row_at<2 * kPe>(lds_qp, lane), row_at<2 * kVal>(lds_y, lane),
                        col_at<2 * kNope>(lds_qn, lane), col_at<2 * kPe>(lds_qp, lane), col_at<2 * kVal>(lds_y, lane),
                        lds_l + 16 * g};
    const float c = a.scale * kLog2e;

    // Queries that do not see the lane's key, or are none.
    const auto hide = [&](int u, f16v &s) {
        if (u >= whole && u < full) return;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int i = u * 32 + 8 * (e / 4) + 4 * g + e % 4;
            s[e] = i >= from && i < sp.lq ? s[e] : -INFINITY;
        }
    };
    if (first < tiles) {
        f16v s0, d0, s1, d1;
        copies_done();
        int st = first % kStages;
#pragma unroll
        for (int n = 0; n < kSdSlots; ++n) {
            const int ks = sd_block(n);
            const uint32_t qn = at.qn + st * (uint32_t)sizeof(sm.qn[0]), qp = at.qp + st * (uint32_t)sizeof(sm.qp[0]);
            if (is_s(n)) {
                const s8 x = ks < kNope / 16 ? row_operand<2 * kNope>(qn, 0, ks) : row_operand<2 * kPe>(qp, 0, ks - kNope / 16);
                if (n == 0) first_product(s0, x, f.k[ks]);
                else add_product(s0, x, f.k[ks]);
            } else {
                const s8 x = row_operand<2 * kVal>(at.y + st * (uint32_t)sizeof(sm.y[0]), 0, ks);
                if (n == 1) first_product(d0, x, f.v[ks]);
                else add_product(d0, x, f.v[ks]);
            }
            if (n % 4 == 3) __builtin_amdgcn_sched_barrier(0);
        }
        products_done();
        for (int t = first; t < tiles - 1; ++t) {
            const int next = st == kStages - 1 ? 0 : st + 1;
            copies_done();  // tile t + 1 is there, and tile t - 1 read
            copy(t + 2);
            hide(2 * t, s0);
            dkv_unit<true>(f, at, st, 0, st, 1, s0, d0, s1, d1, c);
            hide(2 * t + 1, s1);
            dkv_unit<true>(f, at, st, 1, next, 0, s1, d1, s0, d0, c);
            st = next;
        }
        hide(2 * tiles - 2, s0);
        dkv_unit<true>(f, at, st, 0, st, 1, s0, d0, s1, d1, c);
        hide(2 * tiles - 1, s1);
        dkv_unit<false>(f, at, st, 1, 0, 0, s1, d1, s0, d0, c);
    }

    if (SPLIT && tiles_all - first_all > part_tiles) {
#pragma unroll
        for (int d = 0; d < kQk / 32; ++d) leave(part_of<kDkvGroups>(a, place, wave, d), f.dk[d], a.scale);
#pragma unroll
        for (int d = 0; d < kVal / 32; ++d) leave(part_of<kDkvGroups>(a, place, wave, kQk / 32 + d), f.dv[d], 1.0f);
        return;
    }
    __syncthreads();  // the tiles are read
    char *stage = reinterpret_cast<char *>(&sm) + wave * 32 * 2 * kKvRow;
    static_assert(sizeof(sm) >= 4 * 32 * 2 * kKvRow, "");
    const int64_t key = sp.b * a.Tk + sp.k0 + k_first;
#pragma unroll
    for (int d = 0; d < kNope / 32; ++d) stage_values<kKvRow / 8>(stage, lane, 4 * d, f.dk[d], a.scale);
#pragma unroll
    for (int d = 0; d < kVal / 32; ++d) stage_values<kKvRow / 8>(stage, lane, kNope / 8 + 4 * d, f.dv[d], 1.0f);
    store_rows<kKvRow / 8>(stage, lane, a.dkv + (key * a.H + h) * kKvRow, a.H * kKvRow, sp.lk - k_first);
    if (j >= sp.lk) return;
    float *part = a.dpe_part + (h * a.B * a.Tk + key + (lane & 31)) * kPe + 4 * g;
#pragma unroll
    for (int d = 0; d < kPe / 32; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f4 x;
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = f.dk[kNope / 32 + d][4 * e + r] * a.scale;
            *reinterpret_cast<f4 *>(part + 32 * d + 8 * e) = x;
        }
}

__global__ __launch_bounds__(256, 1) void latent_dkv_kernel(LatentArgs a) {
    __shared__ __attribute__((aligned(1024))) DkvSmem sm;
    dkv_block<false>(a, a.base + blockIdx.x, sm);
}

// ---- both at once -------------------------------------------------------------------

// The statistics of every row, 32 a wave, by themselves.
__global__ __launch_bounds__(256) void latent_stat_kernel(LatentArgs a) {
    const int lane = threadIdx.x & 63, g = lane >> 5;
    const int64_t unit = a.base + blockIdx.x, h = unit % a.H, all = a.B * a.T;
    const int64_t t = unit / a.H * kBlock + (threadIdx.x >> 6) * 32 + (lane & 31), at = min(t, all - 1), b = at / a.T, row = at - b * a.T;
    const uint16_t *p = a.dy + b * a.yb + row * a.yt + h * kVal + 8 * g;
    s8 y[kVal / 16];
#pragma unroll
    for (int ks = 0; ks < kVal / 16; ++ks) y[ks] = *reinterpret_cast<const s8 *>(p + 16 * ks);
    const Stat st = row_stat(y, a.o + b * a.ob + row * a.ot + h * kVal + 8 * g, a.lse_in[at * a.H + h]);
    if (g == 0 && t < all) {
        a.stat[h * all + t] = st.lse2;
        a.stat[(a.H + h) * all + t] = st.delta;
    }
}

// The blocks of queries, then those of keys; with SPLIT their parts.
template <bool SPLIT>
__global__ __launch_bounds__(256, 1) void latent_both_kernel(LatentArgs q, LatentArgs k, int64_t q_places) {
    __shared__ __attribute__((aligned(1024))) char sm[sizeof(DkvSmem)];
    static_assert(sizeof(DqSmem) <= sizeof(DkvSmem), "");
    const int64_t place = q.base + blockIdx.x;
    if (place < q_places) dq_block<false, SPLIT>(q, place, *reinterpret_cast<DqSmem *>(sm));
    else dkv_block<SPLIT>(k, place - q_places, *reinterpret_cast<DkvSmem *>(sm));
}

// The parts of a block added up in their order: 32 tokens and 32 of their values a wave.
template <bool BY_KEYS>
__device__ __forceinline__ void join_parts(const LatentArgs &a, int64_t place) {
    constexpr int kGroups = BY_KEYS ? kDkvGroups : kQk / 32;
    const int lane = threadIdx.x, g = lane >> 5;
    const int64_t unit = place / (4 * kGroups), h = unit % a.H;
    const int wave = (int)(place / kGroups % 4), d = (int)(place % kGroups);
    Span sp;
    if (!span_of<kBlock, BY_KEYS>(a, unit / a.H, BY_KEYS ? false : a.causal, sp)) return;
    const int first = sp.block * kBlock, len = BY_KEYS ? sp.lk : sp.lq;
    if (first + wave * 32 >= len) return;
    int tiles;
    if (BY_KEYS) {
        const int from = (a.causal ? max(0, first - (sp.lk - sp.lq)) : 0) / kKeys;
        tiles = (sp.lq + kKeys - 1) / kKeys - from;
    } else {
        const int last = min(sp.lq, first + kBlock) - 1;
        tiles = ((a.causal ? max(0, min(sp.lk, last + 1 + sp.lk - sp.lq)) : sp.lk) + kKeys - 1) / kKeys;
    }
    const int part_tiles = part_tiles_of(a, ((BY_KEYS ? sp.lq : sp.lk) + kKeys - 1) / kKeys);
    if (tiles <= part_tiles) return;
    const int parts = (tiles + part_tiles - 1) / part_tiles;
    f4 v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
        const f4 *x = part_of<kGroups>(a, unit * a.parts + p, wave, d);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += x[e * 64];
    }
    const int i = first + wave * 32 + (lane & 31);
    if (i >= len) return;
    if (BY_KEYS && d >= kNope / 32 && d < kQk / 32) {
        float *part = a.dpe_part + (h * a.B * a.Tk + sp.b * a.Tk + sp.k0 + i) * kPe + 32 * (d - kNope / 32) + 4 * g;
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<f4 *>(part + 8 * e) = v[e];
        return;
    }
    uint16_t *out = BY_KEYS ? a.dkv + ((sp.b * a.Tk + sp.k0 + i) * a.H + h) * kKvRow + 32 * (d < kNope / 32 ? d : d - kPe / 32)
                            : a.dq + ((sp.b * a.T + sp.q0 + i) * a.H + h) * kQk + 32 * d;
#pragma unroll
    for (int e = 0; e < 4; ++e) *reinterpret_cast<u2v *>(out + 4 * g + 8 * e) = u2v{pack2(v[e][0], v[e][1]), pack2(v[e][2], v[e][3])};
}
__global__ __launch_bounds__(64) void latent_grad_join_kernel(LatentArgs q, LatentArgs k, int64_t q_places) {
    const int64_t place = q.base + blockIdx.x;
    if (place < q_places) join_parts<false>(q, place);
    else join_parts<true>(k, place - q_places);
}

// dk_pe: the heads' parts added up, 4 values a thread, heads in order.
__global__ __launch_bounds__(256) void latent_dpe_kernel(const float *part, uint16_t *dpe, const int64_t *cuk, int64_t seqs, int64_t Tk,
                                                         int64_t keys, int64_t H, int64_t base) {
    const int64_t i = (base + blockIdx.x) * 256 + threadIdx.x;
    const int64_t live = cuk ? clamp64(cuk[seqs], 0, Tk) : keys;
    if (i >= live * (kPe / 4)) return;
    const f4 *p = reinterpret_cast<const f4 *>(part) + i;
    const int64_t step = keys * (kPe / 4);
    f4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int64_t h = 0; h < H; ++h) s += p[h * step];
    reinterpret_cast<u2v *>(dpe)[i] = u2v{pack2(s[0], s[1]), pack2(s[2], s[3])};
}

}  // namespace

}  // namespace kda

using namespace kda;

hipError_t kda_launch_latent_pairs(const LatentArgs &q, const LatentArgs &k, hipStream_t s) {
    const int64_t q_units = q.blocks * q.B * q.H, k_units = k.blocks * k.B * k.H;
    // `launch` of a kernel for units, and the arguments with the piece's first one.
    const auto pieces = [&](int64_t units, auto launch) {
        return launch_groups(units, q.launch_cap, [&](int64_t base, dim3 grid) {
            LatentArgs p = q, r = k;
            p.base = r.base = base;
            launch(grid, p, r);
        });
    };
    const dim3 block(256);
    // Where the GPU has a CU for every block of either pass, both run at once, which takes the
    // statistics from a launch ahead (4096 tokens x 4 heads: 241 -> 147 us; 971 x 1: 75 -> 48).
    if (q_units + k_units <= 256) {
        const hipError_t e = pieces((q.B * q.T + kBlock - 1) / kBlock * q.H, [&](dim3 grid, const LatentArgs &p, const LatentArgs &) {
            hipLaunchKernelGGL(latent_stat_kernel, grid, block, 0, s, p);
        });
        if (e != hipSuccess) return e;
        const int64_t q_places = q_units * q.parts, k_places = k_units * k.parts;
        const bool split = q.parts > 1 || k.parts > 1;
        const hipError_t f = pieces(q_places + k_places, [&](dim3 grid, const LatentArgs &p, const LatentArgs &r) {
            if (split) hipLaunchKernelGGL(latent_both_kernel<true>, grid, block, 0, s, p, r, q_places);
            else hipLaunchKernelGGL(latent_both_kernel<false>, grid, block, 0, s, p, r, q_places);
        });
        if (f != hipSuccess || !split) return f;
        const int64_t q_joins = q_units * 4 * (kQk / 32), k_joins = k_units * 4 * kDkvGroups;
        return pieces(q_joins + k_joins, [&](dim3 grid, const LatentArgs &p, const LatentArgs &r) {
            hipLaunchKernelGGL(latent_grad_join_kernel, grid, dim3(64), 0, s, p, r, q_joins);
        });
    }
    const hipError_t e = pieces(q_units, [&](dim3 grid, const LatentArgs &p, const LatentArgs &) {
        hipLaunchKernelGGL(latent_dq_kernel, grid, block, 0, s, p);
    });
    if (e != hipSuccess) return e;
    return pieces(k_units, [&](dim3 grid, const LatentArgs &, const LatentArgs &r) {
        hipLaunchKernelGGL(latent_dkv_kernel, grid, block, 0, s, r);
    });
}

hipError_t kda_launch_latent_dpe(const LatentArgs &a, hipStream_t s) {
    const int64_t keys = a.B * a.Tk;
    return launch_groups((keys * (kPe / 4) + 255) / 256, a.launch_cap, [&](int64_t base, dim3 grid) {
        hipLaunchKernelGGL(latent_dpe_kernel, grid, dim3(256), 0, s, a.dpe_part, a.dpe, a.cu ? a.cuk : nullptr, a.seqs, a.Tk, keys, a.H,
                           base);
    });
}
