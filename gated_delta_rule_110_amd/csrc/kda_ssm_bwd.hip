// kda_ssm_bwd.hip -- the gradient of the selective state-space scan, chunk by
// chunk (gfx950).
//
// The chains of kda_ssm.hip leave, for every chunk of 64 tokens, the state S
// entering it and the gradient D of the state leaving it.  With G, dt and w as
// there, XD_ij = d_out_i . x_j and the masked decays L_ij = e^{G_i - G_j}, j <= i,
//
//   M_ij = L_ij dt_j (C_i . B_j) + [i = j] Dskip,    W_ij = L_ij dt_j XD_ij
//   dx_j = sum_i M_ij d_out_i + w_j D B_j
//   dB_j = sum_i W_ij C_i     + w_j D^T x_j
//   dC_i = sum_j W_ij B_j     + e^{G_i} S^T d_out_i
//
// and with Q_ij = L_ij (C_i . B_j) XD_ij, F_j = w_j x_j^T D B_j, R_i = e^{G_i} d_out_i^T S C_i
// the gradient of a_t collects every pair (i, j) whose decay runs over token t:
//
//   da_t  = e^{G_63} <D, S> + sum_{j < t} F_j + sum_{i >= t} R_i + sum_{i >= t > j} Q_ij dt_j
//   ddt_t = -exp(A_log) da_t + sum_i Q_it + F_t / dt_t,
//
// the double sum, for t in the 16-token tile s, as the column sums of the row tiles
// behind s over j < t, the row sums left of tile s over i >= t in s, and within the
// diagonal tile the rows' sums over j < t added up over i >= t.  (Suffix sums of row
// sum less column sum would be shorter, but pairs behind t cancel there, and the
// rounding of what cancels shows in the gradients of A_log and dt_bias: 1.6e-6 at 12
// tokens, 3.6e-6 over a chunk.)
//
// One workgroup of 8 waves takes a chunk, a group of B and C and a share of its
// heads, one head and 64 channels after the other: C B^T is computed once for
// all of them, and dB and dC add up in registers.  The products' fp32 operands (M, W,
// S, D) are split into three bf16 parts (2^-25); x, B, C and d_out are exact.
//
// What bounds it.  8192 tokens of 64 heads of 64 x 128 take 506 us: 258 here (248, and
// 10 for the sums of shares and parameters), the rest the chains of both directions
// (39 + 41 the pieces, 8 + 9 their joins, 73 + 77 the chunks' states, 268 MB each,
// written at 3.6 TB/s).  One workgroup fits a CU, its waves in step; of 17400 cycles a
// head they spend 3100 on M and W and 1400 waiting for the slowest there, 2500 on dx,
// 8000 on dB and dC, 1500 on staging and the rest in barriers.  LDS is busy for 46% of
// the time, the matrix cores for 24%: latency and LDS reads, not memory (0.45 GB, 1.8
// TB/s).
#include "kda_ssm_common.h"

using namespace kda;

namespace {

constexpr int kThreads = 512;
constexpr int kWaves = 8;
// Rows of x and d_out are read 8 bytes at a time as well as transposed: 16 bytes of
// padding serve the former.
constexpr int kRowPitch = kL + 8;

// M and W (rows i, columns j) hold their 32-column blocks from the diagonal down: 64
// rows of columns 0 to 31, then rows 32 to 63 of the others.  Three parts of both would
// not fit LDS as squares.  A row is 64 bytes, unpadded: its 8-byte groups of columns
// change places by bits 2 and 3 of the row number, so that both the 8-byte and the
// transposing reads of 16 rows spread over the banks.
constexpr int kTriPitch = 32, kTri = 96 * kTriPitch;
// Place of entry (16 it + r, 16 jt + c), where `at` is that of (r, c) in tile (0, 0).
__device__ __forceinline__ int tri_at(int r, int c) { return r * kTriPitch + (c ^ ((r & 4) << 2 | (r & 8))); }
__device__ __forceinline__ int tri_tile(int at, int it, int jt) {
    return (at ^ (jt & 1) << 4) + (16 * it + 16 * (jt & 2)) * kTriPitch;
}

// A head's sums over channels and state entries, shares of its step sizes' gradient.
template <int kN>
struct Sums {
    float colq[4][kL], rowe[2][kL], over[kL], qd[kL], f[4][kL], rr[kN / 16][kL];
    float xs[kN / 16], dd[4];
};

template <int kN>
struct __align__(16) GradSmem {
    uint16_t b[kL * kPitch<kN>], c[kL * kPitch<kN>];
    uint16_t x[kL * kRowPitch], dy[kL * kRowPitch];
    uint16_t m[kParts][kTri], wm[kParts][kTri];        // M and W
    uint16_t d[kParts][kPB * kPitch<kN>];              // D, rows = channels
    Steps s[3];                                        // of the head before, this one and the next
    Sums<kN> sum[2];                                   // of the head before and this one
};

// Operand fragments from LDS.  Along a row: 8 neighbouring entries, or in the
// order of a pair of accumulator tiles (4 g + e, 16 + 4 g + e).  Along rows: by the
// transposing read, in that order too.
__device__ __forceinline__ s8 along(const uint16_t *row, int q, int g) { return lds8(row + 32 * q + 8 * g); }
__device__ __forceinline__ s8 along_pair(const uint16_t *row, int q, int g) {
    return join(*reinterpret_cast<const s4 *>(row + 32 * q + 4 * g), *reinterpret_cast<const s4 *>(row + 32 * q + 16 + 4 * g));
}
__device__ __forceinline__ s8 across(const uint16_t *base, int pitch, int q, int col, int r, int g) {
    const uint16_t *p = base + (32 * q + 4 * g + (r >> 2)) * pitch + col + 4 * (r & 3);
    return join(read_tr(p), read_tr(p + 16 * pitch));
}

// The same of M or W, from the lane's place in a tile: rows 32 q .. of column tile jt, and
// columns 32 q .. of row tile it.
__device__ __forceinline__ s8 tri_across(const uint16_t *base, int at, int q, int jt) {
    const uint16_t *p = base + tri_tile(at, 2 * q, jt);
    return join(read_tr(p), read_tr(p + 16 * kTriPitch));
}
__device__ __forceinline__ s8 tri_along(const uint16_t *base, int at, int it, int q) {
    return join(*reinterpret_cast<const s4 *>(base + tri_tile(at, it, 2 * q)),
                *reinterpret_cast<const s4 *>(base + tri_tile(at, it, 2 * q + 1)));
}

template <int k> struct Int { static constexpr int value = k; };
template <bool k> struct Flag { static constexpr bool value = k; };

// Sum over the 16 lanes of a row, in its last lane.
__device__ __forceinline__ float row16_sum(float v) {
    v += dpp_row_shr_zero(v, 8);
    v += dpp_row_shr_zero(v, 4);
    v += dpp_row_shr_zero(v, 2);
    v += dpp_row_shr_zero(v, 1);
    return v;
}
// Sum over the four 16-lane rows, in every lane: the halves, then the rows, of
// the wave exchanged (lane moves only, no LDS).
__device__ __forceinline__ float rows_sum(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto h = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const float s = __uint_as_float(h[0]) + __uint_as_float(h[1]);
    const uint32_t x = __float_as_uint(s);
    const auto q = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}
// Sum over the 16-lane rows before this lane's (g), of the same place in them.
__device__ __forceinline__ float rows_before(float v, int g) {
    const uint32_t u = __float_as_uint(v);
    const auto q = __builtin_amdgcn_permlane16_swap(u, u, false, false);  // rows 0, 0, 2, 2 and 1, 1, 3, 3
    const float even = __uint_as_float(q[0]);
    const uint32_t x = __float_as_uint(even + __uint_as_float(q[1]));
    const auto h = __builtin_amdgcn_permlane32_swap(x, x, false, false);  // the first half's sum, twice, and the second's
    return (g & 2 ? __uint_as_float(h[0]) : 0.f) + (g & 1 ? even : 0.f);
}
// Sum over the wave, in the last lane of every row.
__device__ __forceinline__ float wave_sum(float v) { return rows_sum(row16_sum(v)); }
// Sum over this lane and those before it.
__device__ __forceinline__ float wave_scan32(float v) {
    auto move = [](float x, auto ctrl, auto rows) {
        return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), decltype(ctrl)::value,
                                                                     decltype(rows)::value, 0xf, false));
    };
    v += move(v, Int<0x111>{}, Int<0xf>{});
    v += move(v, Int<0x112>{}, Int<0xf>{});
    v += move(v, Int<0x114>{}, Int<0xf>{});
    v += move(v, Int<0x118>{}, Int<0xf>{});
    v += move(v, Int<0x142>{}, Int<0xa>{});
    v += move(v, Int<0x143>{}, Int<0xc>{});
    return v;
}
// Sum over this lane and those behind it in its row of 16, in 64 bits.
__device__ __forceinline__ double row_suffix(double v) {
    v += lane_move<0x101, 0xf>(v);
    v += lane_move<0x102, 0xf>(v);
    v += lane_move<0x104, 0xf>(v);
    v += lane_move<0x108, 0xf>(v);
    return v;
}
template <typename T>
__device__ __forceinline__ void add_to(T *p, T v, bool more) { *p = more ? *p + v : v; }

// The same value, as computed here: what follows from it is computed anew rather than kept in
// registers over the loop over the heads, which has none to spare.
__device__ __forceinline__ int here(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// p[i], or 0 without p, by a scalar load; i is the same for the whole wave, and nothing
// here writes the parameters.
__device__ __forceinline__ float scalar(const float *p, int i) {
    typedef const __attribute__((address_space(4))) float cf;
    return p ? reinterpret_cast<cf *>(reinterpret_cast<uintptr_t>(p))[i] : 0.f;
}

// The derivative of softplus, from its value dt: 1 - e^-dt, for small dt by its series
// (to dt^8: the next term is below 2^-25 relative at 1/2).
__device__ __forceinline__ float softplus_slope(float dt) {
    float s = -1.0f / 8.0f;
    s = __builtin_fmaf(s, dt, 1.0f) * (1.0f / 7.0f);
    s = __builtin_fmaf(-s, dt, 1.0f) * (1.0f / 6.0f);
    s = __builtin_fmaf(-s, dt, 1.0f) * (1.0f / 5.0f);
    s = __builtin_fmaf(-s, dt, 1.0f) * (1.0f / 4.0f);
    s = __builtin_fmaf(-s, dt, 1.0f) * (1.0f / 3.0f);
    s = __builtin_fmaf(-s, dt, 1.0f) * (1.0f / 2.0f);
    s = __builtin_fmaf(-s, dt, 1.0f) * dt;
    return dt < 0.5f ? s : 1.0f - exact_exp(-dt);
}

// Tokens of chunk number i of the batch.
struct Chunk {
    int64_t row0, t0;
    int rows;
};
__device__ __forceinline__ bool chunk_of(const SsmGradArgs &a, int64_t i, Chunk &c) {
    int64_t begin = 0, len = a.T, k;
    if (a.cu) {
        if (i >= a.chunk_off[a.seqs]) return false;
        const int64_t n = seq_of_slot(a.chunk_off, a.seqs, i);
        k = i - a.chunk_off[n];
        begin = clamp_to(a.cu[n], a.T);
        len = clamp_to(a.cu[n + 1], a.T) - begin;
        c.row0 = 0;
    } else {
        if (i >= a.seqs * a.cps) return false;
        c.row0 = i / a.cps;
        k = i - c.row0 * a.cps;
    }
    c.t0 = begin + k * kL;
    const int64_t left = len - k * kL;
    c.rows = (int)(left < kL ? left : kL);
    return c.rows > 0;
}

template <int kN>
__global__ __launch_bounds__(kThreads) void kda_ssm_grad_kernel(SsmGradArgs a) {
    constexpr int kTiles = kN / 16, kQ = kN / 32;
    constexpr int kJ = 4 * kTiles / kWaves;      // token tiles of dB and dC per wave
    __shared__ GradSmem<kN> sm;
    const int64_t per = a.G * a.shares;
    const int64_t block = a.base + blockIdx.x;
    const int64_t chunk = block / per;
    const int64_t grp = (block - chunk * per) / a.shares;
    const int share = (int)(block - chunk * per - grp * a.shares);
    Chunk ck;
    if (chunk >= a.chunks || !chunk_of(a, chunk, ck)) return;
    const int rows = ck.rows;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int it = w & 3, kb = w >> 2;           // this wave's tiles of the 64 x 64 products
    const int nt = w % kTiles, j0 = kTiles < kWaves ? w / kTiles * kJ : 0;
    const int along_at = tri_at(r, 4 * g), across_at = tri_at(4 * g + (r >> 2), 4 * (r & 3));  // in M and W
    const int H = (int)a.H, heads = H / (int)a.G;  // of the group
    const int h0 = (int)grp * heads + share * a.share;
    const int count = heads - share * a.share < a.share ? heads - share * a.share : a.share;
    const int pbs = a.P == 2 * kPB ? 2 : 1, shift = pbs - 1;
    const uint16_t *xrow = a.x + ck.row0 * a.xb + ck.t0 * a.xt;
    const uint16_t *yrow = a.dy + ck.row0 * a.yb + ck.t0 * a.yt;
    const int64_t trow = ck.row0 * a.T + ck.t0;  // row of the contiguous outputs

    {
        Rows<kN, kThreads> rb, rc;
        rb.init(a.bt, kPitch<kN>);
        rc.init(a.ct, kPitch<kN>);
        rb.load(a.Bm + ck.row0 * a.bb + ck.t0 * a.bt + grp * kN, rows);
        rc.load(a.Cm + ck.row0 * a.cb + ck.t0 * a.ct + grp * kN, rows);
        rb.store(sm.b, kPitch<kN>);
        rc.store(sm.c, kPitch<kN>);
    }
    __syncthreads();
    f4 cb[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};  // (C_i . B_j): lane = i, entries j
    if (2 * kb <= it) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int q = 0; q < kQ; ++q)
                cb[half] = mfma16x16x32_bf16(along(sm.b + (32 * kb + 16 * half + r) * kPitch<kN>, q, g),
                                             along(sm.c + (16 * it + r) * kPitch<kN>, q, g), cb[half]);
    }
    if (kb == 0 && it < 2) {                     // tiles (0, 1) and (2, 3) of M and W are zero
        float none[4] = {0.f, 0.f, 0.f, 0.f};
        const int at = tri_tile(along_at, 2 * it, 2 * it + 1);
        keep_parts(none, &sm.m[0][at], kTri);
        keep_parts(none, &sm.wm[0][at], kTri);
    }
    f4 dB[kJ], dC[kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) dB[j] = dC[j] = f4{0.f, 0.f, 0.f, 0.f};

    // The next head's (or channel block's) tensors are loaded while one is computed;
    // barriers order LDS traffic only, so that the loads stay in flight across them.
    constexpr int kPairs = kN / 64;              // pairs of D's tiles per thread, 8 neighbouring entries each
    const int dq = w % kQ, dp = w / kQ;
    const int units = count << shift;
    Rows<kPB, kThreads> rx, ry;
    rx.init(a.xt, kRowPitch);
    ry.init(a.yt, kRowPitch);
    f4 D[2 * kPairs], S[4];
    constexpr int kRows = 1, kD = 2, kS = 4, kAll = 7;
    auto fetch = [&](int u, const int what) {
        if (u >= units) return;
        const int h = h0 + (u >> shift), pb = u & shift;
        const int64_t unit = ((chunk * H + h) << shift) + pb;
        const f4 *hs = reinterpret_cast<const f4 *>(a.hs) + unit * (kPB * kN / 4);
        const f4 *ds = reinterpret_cast<const f4 *>(a.ds) + unit * (kPB * kN / 4);
        if (what & kRows) {
            rx.load(xrow + ((h << shift) + pb) * kPB, rows);
            ry.load(yrow + ((h << shift) + pb) * kPB, rows);
        }
        if (what & kD)
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) D[2 * i + k] = ds[((dp + i * (kWaves / kQ)) * kTiles + 2 * dq + k) * 64 + lane];
        // rows = channels 16 t + 4 g + e, column = entry 16 nt + r
        if (what & kS)
#pragma unroll
            for (int t = 0; t < 4; ++t) S[t] = hs[(t * kTiles + nt) * 64 + lane];
    };
    // The work per token of a head, lane = token: its step sizes ahead of its
    // turn, and the sums' gradients behind it, each by a wave that the 64 x 64
    // products leave idle.
    // Parameters come by scalar loads, and the raw step sizes a head ahead: waits for
    // vector loads are in order, and one within the products would wait for the rows
    // just fetched.
    // Lanes and heads behind the last ones read those again.
    const uint16_t *drow = a.dt + ck.row0 * a.dtb + (ck.t0 + (lane < rows ? lane : rows - 1)) * a.dtt + h0;
    auto raw_of = [&](int i) -> uint32_t { return drow[i < count ? i : count - 1]; };
    auto steps_of = [&](int i, uint32_t raw, Steps &to) {
        step_sizes(bf16_bits_to_f32((uint16_t)raw), lane < rows, scalar(a.dt_bias, h0 + i),
                   -decay_rate(scalar(a.A_log, h0 + i)) * kLog2e, to);
    };
    auto finish = [&](int i, const Steps &st, const Sums<kN> &su) {
        const float A = -decay_rate(scalar(a.A_log, h0 + i));
        const int t = lane;
        float cq[4], colq = 0.f, f = 0.f, rr = 0.f, xs = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = su.colq[i][t];       // row tiles before t's hold none
            cq[i] = i >= t >> 4 ? v : 0.f;
            colq += cq[i];
            f += su.f[i][t];
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            rr += su.rr[i][t];
            xs += su.xs[i];
        }
        const float gl = st.g[kL - 1], glr = st.gr[kL - 1], dt = st.dt[t];
        const float wd = __builtin_amdgcn_exp2f((gl - st.g[t]) + (glr - st.gr[t]));
        rr *= st.from[t];
        xs *= st.from[kL - 1];
        const double z = rr, F = (double)wd * (double)dt * (double)f;
        const double zi = wave_scan(z), fi = wave_scan(F);
        const double total = __shfl(zi, 63);
        const int tile = t >> 4;
        const double rows_left = row_suffix((double)su.rowe[0][t] + (double)(t >= 32 ? su.rowe[1][t] : 0.f));
        float left = 0.f;
#pragma unroll
        for (int i = 1; i < 4; ++i) {            // row tiles behind t's, columns before t: nothing cancels
            const float v = tile < i ? dt * cq[i] : 0.f;
            const float before = wave_scan32(v) - v;
            left += tile < i ? before : 0.f;
        }
        const float da = (float)((double)xs + (fi - F) + (total - zi + z) + (rows_left + (double)left + (double)su.over[t]));
        const float ddt = A * da + (colq + su.qd[t]) + wd * f;
        const float draw = t < rows ? ddt * softplus_slope(dt) : 0.f;
        if (t < rows) a.ddt[(trow + t) * H + h0 + i] = f32_to_bf16_bits(draw);
        const float dA = wave_sum(A * dt * da), db = wave_sum(draw);
        if (lane == 63) {
            float *p = a.psum + (chunk * H + h0 + i) * 4;
            p[0] = dA;
            p[1] = db;
            p[2] = (su.dd[0] + su.dd[1]) + (su.dd[2] + su.dd[3]);
        }
    };
    constexpr int kFinisher = 4, kStepper = 5;   // waves without a tile below the diagonal
    uint32_t raw = 0;                            // the stepper's, of the next head
    if (w == kStepper) {
        steps_of(0, raw_of(0), sm.s[0]);
        raw = raw_of(1);
    }
    fetch(0, kAll);
    int slot = 0;                                // of this head's step sizes
    for (int u = 0; u < units; ++u) {
        const int i = u >> shift, h = h0 + i, pb = u & shift;
        const float Dh = scalar(a.D, h);
        const bool more = pb > 0;                // sums over channels go on
        if (u > 0 && !more) slot = slot == 2 ? 0 : slot + 1;
        const Steps &st = sm.s[slot];
        Sums<kN> &su = sm.sum[i & 1];
        {
            rx.store(sm.x, kRowPitch);
            ry.store(sm.dy, kRowPitch);
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = D[2 * i][e];
                    v[4 + e] = D[2 * i + 1][e];
                }
                s8 d0, d1, d2;
                split3(v, d0, d1, d2);
                const int at = (16 * (dp + i * (kWaves / kQ)) + r) * kPitch<kN> + 32 * dq + 8 * g;
                *reinterpret_cast<s8 *>(&sm.d[0][at]) = d0;
                *reinterpret_cast<s8 *>(&sm.d[1][at]) = d1;
                *reinterpret_cast<s8 *>(&sm.d[2][at]) = d2;
            }
            asm volatile("" : "+v"(raw));       // waited for here, before the rows' loads
            lds_barrier();
            fetch(u + 1, kRows);

            // ---- M, W, Q: 64 x 64, lane = i, entries j
            if (w == kFinisher && !more) {
                if (i > 0) finish(i - 1, sm.s[slot == 0 ? 2 : slot - 1], sm.sum[(i - 1) & 1]);
            }
            if (w == kStepper && !more && i + 1 < count) {
                steps_of(i + 1, raw, sm.s[slot == 2 ? 0 : slot + 1]);
                raw = raw_of(i + 2);
            }
            if (2 * kb <= it) {
                const int ti = 16 * it + r;
                const float gi = st.g[ti], gir = st.gr[ti];
                // One 16 x 16 tile; the sums are returned: of the row, and in the diagonal
                // tile of Q and of XD at i = j.
                auto tile = [&](const int half, auto on_diagonal, float &row, float &qd, float &dd) {
                    constexpr bool kDiagonal = decltype(on_diagonal)::value;
                    const int jt = 2 * kb + half;
                    f4 xd = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        xd = mfma16x16x32_bf16(along(sm.x + (16 * jt + r) * kRowPitch, q, g), along(sm.dy + ti * kRowPitch, q, g), xd);
                    const f4 gj = *reinterpret_cast<const f4 *>(&st.g[16 * jt + 4 * g]);
                    const f4 rj = *reinterpret_cast<const f4 *>(&st.gr[16 * jt + 4 * g]);
                    const f4 dj = *reinterpret_cast<const f4 *>(&st.dt[16 * jt + 4 * g]);
                    float m[4], wv[4];
                    [[maybe_unused]] float pair[4];
                    f4 col;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int tj = 16 * jt + 4 * g + e;
                        float l = __builtin_amdgcn_exp2f((gi - gj[e]) + (gir - rj[e]));
                        if (kDiagonal) l = tj <= ti ? l : 0.f;
                        const float lc = l * cb[half][e];
                        float qv = lc * xd[e];
                        m[e] = lc * dj[e];
                        wv[e] = l * dj[e] * xd[e];
                        if (kDiagonal) {
                            // lanes above the diagonal: 0 times what is there could be NaN
                            const bool is = tj == ti;
                            m[e] = tj <= ti ? m[e] + (is ? Dh : 0.f) : 0.f;
                            wv[e] = tj <= ti ? wv[e] : 0.f;
                            qd += is ? qv : 0.f;
                            dd += is ? xd[e] : 0.f;
                            qv = tj < ti ? qv : 0.f;
                        }
                        if (kDiagonal) pair[e] = qv * dj[e];
                        else row += qv * dj[e];
                        col[e] = row16_sum(qv);
                    }
                    if constexpr (kDiagonal) {
                        // for every t in the tile: each row's sum over j < t, then the rows i >= t
                        float before = rows_before(((pair[0] + pair[1]) + pair[2]) + pair[3], g);
                        f4 over;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            over[e] = row16_sum(4 * g + e <= r ? before : 0.f);
                            before += pair[e];
                        }
                        if (r == 15) add_to(reinterpret_cast<f4 *>(&su.over[16 * jt + 4 * g]), over, more);
                    }
                    if (r == 15) add_to(reinterpret_cast<f4 *>(&su.colq[it][16 * jt + 4 * g]), col, more);
                    const int at = tri_tile(along_at, it, jt);
                    keep_parts(m, &sm.m[0][at], kTri);
                    keep_parts(wv, &sm.wm[0][at], kTri);
                };
                float rowe = 0.f, qd = 0.f, dd = 0.f, none = 0.f;
                if (it == 2 * kb) {
                    tile(0, Flag<true>{}, none, qd, dd);
                } else if (it == 2 * kb + 1) {
                    tile(0, Flag<false>{}, rowe, none, none);
                    tile(1, Flag<true>{}, none, qd, dd);
                } else {
                    tile(0, Flag<false>{}, rowe, none, none);
                    tile(1, Flag<false>{}, rowe, none, none);
                }
                rowe = rows_sum(rowe);
                if (g == 0) add_to(&su.rowe[kb][ti], rowe, more);
                if (kb == it >> 1) {             // the wave with the diagonal tile
                    dd = wave_sum(dd);
                    if (lane == 63) add_to(&su.dd[it], dd, more);
                    if (g == r >> 2) add_to(&su.qd[ti], qd, more);
                }
            }
            fetch(u + 1, kD);
            lds_barrier();

            // ---- dx, transposed: lane = token, entries 4 neighbouring channels
            {
                const int pt = w & 3, half = w >> 2;
                // both token tiles side by side, the parts in accumulators of their own: four
                // products between any two of one chain
                f4 u[2][2];
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) u[jj][0] = u[jj][1] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < kQ; ++q) {
                    const s8 d0 = along(sm.d[0] + (16 * pt + r) * kPitch<kN>, q, g), d1 = along(sm.d[1] + (16 * pt + r) * kPitch<kN>, q, g),
                             d2 = along(sm.d[2] + (16 * pt + r) * kPitch<kN>, q, g);
#pragma unroll
                    for (int jj = 0; jj < 2; ++jj) {
                        const s8 bv = along(sm.b + (32 * half + 16 * jj + r) * kPitch<kN>, q, g);
                        u[jj][0] = mfma16x16x32_bf16(d0, bv, u[jj][0]);
                        u[jj][1] = mfma16x16x32_bf16(d1, bv, u[jj][1]);
                        u[jj][1] = mfma16x16x32_bf16(d2, bv, u[jj][1]);
                    }
                }
                float fs[2];
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    const int tj = 32 * half + 16 * jj + r;
                    const s4 xv = *reinterpret_cast<const s4 *>(sm.x + tj * kRowPitch + 16 * pt + 4 * g);
                    float f = 0.f;
                    const float wj = st.w[tj];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float v = u[jj][0][e] + u[jj][1][e];
                        f += bf16_bits_to_f32((uint16_t)xv[e]) * v;
                        u[jj][0][e] = v * wj;
                        u[jj][1][e] = 0.f;
                    }
                    fs[jj] = rows_sum(f);
                }
#pragma unroll
                for (int jj = 0; jj < 2; ++jj)
                    if (g == 0) add_to(&su.f[pt][32 * half + 16 * jj + r], fs[jj], more);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (q < half) continue;      // i before j
                    const s8 yv = across(sm.dy, kRowPitch, q, 16 * pt, r, g);
#pragma unroll
                    for (int k = 0; k < kParts; ++k)
#pragma unroll
                        for (int jj = 0; jj < 2; ++jj)
                            u[jj][k > 0] = mfma16x16x32_bf16(yv, tri_across(sm.m[k], across_at, q, 2 * half + jj), u[jj][k > 0]);
                }
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    const int tj = 32 * half + 16 * jj + r;
                    const f4 v = u[jj][0] + u[jj][1];
                    if (tj < rows)
                        *reinterpret_cast<uint2 *>(a.dx + ((((trow + tj) * H + h) << shift) + pb) * kPB + 16 * pt + 4 * g) =
                            make_uint2(pack_pair(v[0], v[1]), pack_pair(v[2], v[3]));
                }
            }

            // ---- dB and dC, transposed: lane = token, entries 4 neighbouring state entries; one
            // after the other, so that D's parts and S's are not held together
            {
                s8 Dv[kParts][2], Ct[2];
                float xs = 0.f;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    Ct[q] = across(sm.c, kPitch<kN>, q, 16 * nt, r, g);
#pragma unroll
                    for (int k = 0; k < kParts; ++k) Dv[k][q] = across(sm.d[k], kPitch<kN>, q, 16 * nt, r, g);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        xs += S[2 * q + (e >> 2)][e & 3] *
                              (bf16_bits_to_f32((uint16_t)Dv[0][q][e]) +
                               (bf16_bits_to_f32((uint16_t)Dv[1][q][e]) + bf16_bits_to_f32((uint16_t)Dv[2][q][e])));
                }
                xs = wave_sum(xs);
                if (lane == 63 && j0 == 0) add_to(&su.xs[nt], xs, more);
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    const int tt = j0 + j, t = 16 * tt + r;
                    f4 u = {0.f, 0.f, 0.f, 0.f}, v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const s8 xv = along_pair(sm.x + t * kRowPitch, q, g);
                        u = mfma16x16x32_bf16(Dv[0][q], xv, u);
                        v = mfma16x16x32_bf16(Dv[1][q], xv, v);
                        v = mfma16x16x32_bf16(Dv[2][q], xv, v);
                    }
                    const float wt = st.w[t];
#pragma unroll
                    for (int e = 0; e < 4; ++e) dB[j][e] += wt * (u[e] + v[e]);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        if (2 * q + 1 < tt) continue;  // i from token tile tt on
#pragma unroll
                        for (int k = 0; k < kParts; ++k)
                            dB[j] = mfma16x16x32_bf16(Ct[q], tri_across(sm.wm[k], across_at, q, tt), dB[j]);
                    }
                }
            }
            {
                const int own = here(lane), r = own & 15, g = own >> 4;
                const int along_at = tri_at(r, 4 * g);
                s8 Sv[kParts][2], Bt[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    Bt[q] = across(sm.b, kPitch<kN>, q, 16 * nt, r, g);
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = S[2 * q + (e >> 2)][e & 3];
                    split3(v, Sv[0][q], Sv[1][q], Sv[2][q]);
                }
                fetch(u + 1, kS);
                float rr[kJ];
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    const int tt = j0 + j, t = 16 * tt + r;
                    f4 u = {0.f, 0.f, 0.f, 0.f}, v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const s8 yv = along_pair(sm.dy + t * kRowPitch, q, g);
                        u = mfma16x16x32_bf16(Sv[0][q], yv, u);
                        v = mfma16x16x32_bf16(Sv[1][q], yv, v);
                        v = mfma16x16x32_bf16(Sv[2][q], yv, v);
                    }
                    const s4 cv = *reinterpret_cast<const s4 *>(sm.c + t * kPitch<kN> + 16 * nt + 4 * g);
                    const float et = st.from[t];
                    float f = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float s = u[e] + v[e];
                        f += bf16_bits_to_f32((uint16_t)cv[e]) * s;
                        dC[j][e] += et * s;
                    }
                    rr[j] = rows_sum(f);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        if (2 * q > tt) continue;      // j up to token tile tt
#pragma unroll
                        for (int k = 0; k < kParts; ++k)
                            dC[j] = mfma16x16x32_bf16(Bt[q], tri_along(sm.wm[k], along_at, tt, q), dC[j]);
                    }
                }
#pragma unroll
                for (int j = 0; j < kJ; ++j)
                    if (g == 0) add_to(&su.rr[nt][16 * (j0 + j) + r], rr[j], more);
            }
            lds_barrier();
        }
    }
    if (w == kFinisher) finish(count - 1, sm.s[slot], sm.sum[(count - 1) & 1]);

#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        const int t = 16 * (j0 + j) + r, n = 16 * nt + 4 * g;
        if (t >= rows) continue;
        if (a.shares == 1) {
            const int64_t o = ((trow + t) * a.G + grp) * kN + n;
            *reinterpret_cast<uint2 *>(a.dB + o) = make_uint2(pack_pair(dB[j][0], dB[j][1]), pack_pair(dB[j][2], dB[j][3]));
            *reinterpret_cast<uint2 *>(a.dC + o) = make_uint2(pack_pair(dC[j][0], dC[j][1]), pack_pair(dC[j][2], dC[j][3]));
        } else {
            const int64_t one = a.chunks * a.G * kL * kN;  // a share of one of the two
            const int64_t o = ((chunk * a.G + grp) * kL + t) * kN + n;
            *reinterpret_cast<f4 *>(a.part + share * one + o) = dB[j];
            *reinterpret_cast<f4 *>(a.part + (a.shares + share) * one + o) = dC[j];
        }
    }
}

// dB and dC from the shares, in order: kJoin workgroups per chunk and group, for
// dB (the first half of them) and dC.
constexpr int kJoin = 8;

template <int kN>
__global__ __launch_bounds__(256) void kda_ssm_grad_join_kernel(SsmGradArgs a) {
    const int64_t place = a.base + blockIdx.x, block = place / kJoin;
    const int64_t chunk = block / a.G, grp = block - chunk * a.G;
    Chunk ck;
    if (chunk >= a.chunks || !chunk_of(a, chunk, ck)) return;
    const int part = (int)(place % kJoin), which = part / (kJoin / 2);
    const int64_t one = a.chunks * a.G * kL * kN;
    const float *from = a.part + which * a.shares * one + (chunk * a.G + grp) * kL * kN;
    uint16_t *to = (which ? a.dC : a.dB) + ((ck.row0 * a.T + ck.t0) * a.G + grp) * kN;
    for (int i = (part % (kJoin / 2)) * 256 + threadIdx.x; i < ck.rows * kN / 4; i += kJoin / 2 * 256) {
        const int t = i / (kN / 4), n = 4 * (i % (kN / 4));
        const float *src = from + t * kN + n;
        f4 v = *reinterpret_cast<const f4 *>(src);
        for (int s = 1; s < a.shares; ++s) v += *reinterpret_cast<const f4 *>(src + s * one);
        *reinterpret_cast<uint2 *>(to + t * a.G * kN + n) = make_uint2(pack_pair(v[0], v[1]), pack_pair(v[2], v[3]));
    }
}

// dA_log, ddt_bias and dD: the chunks' sums, in a fixed order and in 64 bits.
__global__ __launch_bounds__(256) void kda_ssm_grad_params_kernel(SsmGradArgs a) {
    __shared__ double s[3][256];
    const int64_t h = blockIdx.x;
    const int64_t chunks = a.cu ? clamp_to(a.chunk_off[a.seqs], a.chunks) : a.chunks;
    double v[3] = {0.0, 0.0, 0.0};
    for (int64_t c = threadIdx.x; c < chunks; c += 256)
#pragma unroll
        for (int k = 0; k < 3; ++k) v[k] += (double)a.psum[(c * a.H + h) * 4 + k];
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k][threadIdx.x] = v[k];
    __syncthreads();
    for (int d = 128; d >= 1; d >>= 1) {
        if ((int)threadIdx.x < d)
#pragma unroll
            for (int k = 0; k < 3; ++k) s[k][threadIdx.x] += s[k][threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        a.dA_log[h] = (float)s[0][0];
        if (a.ddt_bias) a.ddt_bias[h] = (float)s[1][0];
        if (a.dD) a.dD[h] = (float)s[2][0];
    }
}

template <int kN>
hipError_t launch(const SsmGradArgs &a, hipStream_t s) {
    if (a.chunks > 0 && a.T > 0) {
        SsmGradArgs b = a;
        // its workgroups have twice the threads that launch_groups counts with
        const int64_t cap = launch_piece(int64_t(1) << 22, a.launch_cap);
        hipError_t e = launch_groups(a.chunks * a.G * a.shares, cap, [&](int64_t base, dim3 grid) {
            b.base = base;
            hipLaunchKernelGGL((kda_ssm_grad_kernel<kN>), grid, dim3(kThreads), 0, s, b);
        });
        if (e == hipSuccess && a.shares > 1)
            e = launch_groups(a.chunks * a.G * kJoin, a.launch_cap, [&](int64_t base, dim3 grid) {
                b.base = base;
                hipLaunchKernelGGL((kda_ssm_grad_join_kernel<kN>), grid, dim3(256), 0, s, b);
            });
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kda_ssm_grad_params_kernel, dim3((unsigned)a.H), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t kda_launch_ssm_grad(const SsmGradArgs &a, int N, hipStream_t s) {
    return N == 128 ? launch<128>(a, s) : launch<64>(a, s);
}
