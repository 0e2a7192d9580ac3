// kda_ssm.hip -- the selective state-space scan over whole sequences (gfx950).
//
// In chunks of 64 tokens, with a_t = -exp(A_log) dt_t and G_i = sum_{t <= i} a_t
// within the chunk, the recurrence S_t = e^{a_t} S_{t-1} + dt_t x_t B_t^T becomes
//
//   y_i   = e^{G_i} S C_i + sum_{j <= i} M_ij x_j,   M_ij = e^{G_i - G_j} dt_j (C_i . B_j) + [i = j] D
//   S     <- e^{G_63} S + sum_j w_j x_j B_j^T,        w_j  = e^{G_63 - G_j} dt_j
//
// four products on the matrix cores per chunk and head (C B^T, M x, C S^T, the
// update), with every decay at most 1, so that nothing overflows.
//
// x, B and C are bf16, exact as operands.  What is computed in fp32 and then
// needed as an operand (M, S, the weighted x) is split into three bf16 parts,
// together 2^-25, half of fp32's own step: the products are those of fp32.  States,
// decays and sums stay in fp32.
//
// What bounds it.  8192 tokens of 64 heads of 64 x 128 take 127 us (39 for the pieces'
// states, 8 to join them, 80 for the outputs), where the tensors alone would take 23:
// the products, in parts, are 90 GFLOP, 40 us of the matrix cores at the clock they
// run at here, and a chunk's four products, its 64 decays and two barriers follow one
// another.  Per chunk and wave the outputs' pass spends 10400 cycles: 2000 on C S^T and
// 2200 on the update, both near the matrix cores' rate with two workgroups a CU, 2700
// on M and 1600 on M x, which wait for LDS and for each other, 1900 on staging, stores
// and barriers.  32768 packed tokens of 32 heads of 128 x 128: 481 us; 131072 tokens of
// 4 heads of 64 x 64: 99 us.
//
// Work.  Chains are serial over chunks but independent over heads and over
// blocks of 64 channels, and 64 x N states leave most of the GPU idle for a
// single prompt; so sequences are cut into pieces: a first pass walks through
// each piece from a zero state (kPieces: B and x only), a scan joins the states
// of the pieces in fp32, and the second pass starts each piece from the state
// that enters it.  With one piece per sequence only the last pass runs.
//
// A workgroup of four waves holds the state of 64 channels in registers, 16
// channels a wave: S^T as MFMA accumulators, tile t of 16 state rows by the
// wave's channels, rows numbered so that a pair of tiles is at once the operand
// of the next product (rows 4 g + e of tiles 2 q and 2 q + 1 stand for n = 32 q +
// 8 g + e and + 4).  B, C and x of the chunk are staged in LDS row by row; the
// operands that run along tokens are read back with the transposing LDS read.
#include "kda_ssm_common.h"

using namespace kda;

namespace {

constexpr int kThreads = 256;

// Passes over a piece.
constexpr int kPieces = 0;    // from zero: the piece's own state and its decay
constexpr int kOutputs = 1;   // outputs and final states
constexpr int kSave = 2;      // the state entering every chunk, for the gradient
constexpr int kStepper = 3;   // the wave that takes the step sizes

// One piece: its sequence, tokens and place.
struct Piece {
    int64_t n, slot;           // sequence; slot of the piece's state, where the sequence has several
    int64_t row0, t0;          // batch row and token of its first token
    int count;                 // tokens
    int64_t chunk0;            // number of its first chunk in the batch
    bool first, last;          // of its sequence
    bool valid;
};

__device__ __forceinline__ Piece piece_of(const SsmChainArgs &a, int64_t index) {
    Piece p;
    p.slot = index;
    p.valid = false;
    int64_t begin = 0, len = a.T, k, per = a.pc;
    if (index >= a.pieces) return p;
    if (a.cu) {
        if (index >= a.piece_off[a.seqs]) return p;
        p.n = seq_of_slot(a.piece_off, a.seqs, index);
        k = index - a.piece_off[p.n];
        begin = clamp_to(a.cu[p.n], a.T);
        len = clamp_to(a.cu[p.n + 1], a.T) - begin;
        if (len <= 0) return p;
        // as many pieces as of pc chunks, but even ones (1 to 3% less time than with a rest)
        const uint32_t chunks = (uint32_t)((len + kL - 1) / kL);
        const uint32_t pieces = (chunks + (uint32_t)a.pc - 1) / (uint32_t)a.pc;
        per = (chunks + pieces - 1) / pieces;
        p.slot = a.slot_off[p.n] + k;
        if (pieces > 1 && p.slot >= a.slots) return p;  // lengths that no batch has
        p.row0 = 0;
        p.chunk0 = a.chunk_off[p.n] + k * per;
    } else {
        p.n = index / a.pps;
        k = index - p.n * a.pps;
        p.row0 = p.n;
        p.chunk0 = p.n * a.cps + k * per;
    }
    const int64_t from = k * per * kL, size = per * kL;
    p.t0 = begin + from;
    p.count = (int)(len - from < size ? len - from : size);
    p.first = k == 0;
    p.last = from + size >= len;
    p.valid = p.count > 0;
    return p;
}

// Workgroups to (piece, head, channel block).  Workgroups go to the 8 XCDs in turn.
// Each XCD gets an eighth of the heads, of all pieces, so that uneven pieces load
// them evenly; with a number of heads that is no multiple of 8 it gets whole pieces.
// Either way the heads that share B and C find them in its L2.
__device__ __forceinline__ void place(const SsmChainArgs &a, int64_t &piece, int64_t &h, int64_t &pb) {
    const int64_t units = a.H * (a.P / kPB);
    const int64_t i = (a.base + blockIdx.x) >> 3, xcd = blockIdx.x & 7;
    int64_t u;
    if (units % 8 == 0) {
        const int64_t own = units / 8;
        piece = i / own;
        u = xcd * own + (i - piece * own);
    } else {
        u = i % units;
        piece = (i / units) * 8 + xcd;
    }
    h = u / (a.P / kPB);
    pb = u - h * (a.P / kPB);
}
int64_t grid_size(const SsmChainArgs &a) {
    const int64_t units = a.H * (a.P / kPB);
    return (units % 8 == 0 ? a.pieces : (a.pieces + 7) / 8 * 8) * units;
}

// The decays that M's tiles left of the diagonal take as products around their
// row tile's first token, both factors at most 1.
struct TileDecays {
    float upto[kL];               // from the token before the row tile to token i
    float before[3][kL];          // from token j to the token before row tile 1, 2, 3, times dt_j
};

template <int kN, bool kOut>
struct __align__(16) ChainSmem {
    uint16_t k[kL * kPitch<kN>];
    uint16_t c[kOut ? kL * kPitch<kN> : 8];
    uint16_t x[kL * kXPitch];                   // and then the chunk's outputs, on their way to whole rows
    uint16_t m[kOut ? kParts * 4 * 2 * 64 * 8 : 8];  // M as operands: [part][row tile][k block][lane][8]
    Steps s[2];                                 // of this chunk and the next
    TileDecays t[kOut ? 2 : 1];
    int special;                                // outputs to be taken again
};

// By the wave that wrote the steps, lane = token, from what the lane itself wrote and
// the tokens before the row tiles (a wave's own LDS accesses are in order).
__device__ __forceinline__ void tile_decays(const Steps &s, TileDecays &o) {
    const int lane = threadIdx.x & 63;
    const float g = s.g[lane], gr = s.gr[lane], dt = s.dt[lane];
    float up = 1.f;
#pragma unroll
    for (int it = 1; it < 4; ++it) {
        const float g0 = s.g[16 * it - 1], g0r = s.gr[16 * it - 1];
        // tokens of the tile and behind it: not read, kept finite
        o.before[it - 1][lane] = lane < 16 * it ? __builtin_amdgcn_exp2f((g0 - g) + (g0r - gr)) * dt : 0.f;
        if (lane >= 16 * it) up = __builtin_amdgcn_exp2f((g - g0) + (gr - g0r));
    }
    o.upto[lane] = up;
}

// 8 consecutive state entries of either type.
__device__ __forceinline__ void load_state8(const void *p, int64_t i, int f32, float *o) {
    if (f32) {
        const float4 a = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p) + i);
        const float4 b = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p) + i + 4);
        o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
        o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
    } else {
        unpack_bf16x8(*reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(p) + i), o);
    }
}
__device__ __forceinline__ void store_state8(void *p, int64_t i, int f32, const f4 &lo, const f4 &hi) {
    if (f32) {
        float *q = reinterpret_cast<float *>(p) + i;
        *reinterpret_cast<f4 *>(q) = lo;
        *reinterpret_cast<f4 *>(q + 4) = hi;
    } else {
        *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(p) + i) =
            make_uint4(pack_bf16(lo[0], lo[1]), pack_bf16(lo[2], lo[3]), pack_bf16(hi[0], hi[1]), pack_bf16(hi[2], hi[3]));
    }
}

// NaN and infinities in x.  M's zeros above the diagonal carry them to the tokens
// before, as products of M x do, and to every token of the chunk's last tile, where a
// test of 4 values a lane finds them.  A piece with any there is walked through again,
// its waves then leaving them out of M x and adding their products to the tokens from
// theirs on one by one.  (Doing so at once, behind a test of x, put branches into every
// chunk: a packed prompt of 32768 tokens x 32 heads 487 us, this way 473, without 464.)
__device__ __forceinline__ bool is_special(uint32_t bits16) { return (bits16 & 0x7f80u) == 0x7f80u; }
__device__ __forceinline__ bool any_special(const s8 (&x)[2]) {
    uint32_t full = 0;                           // bit 15 of a half: its exponent has all bits set
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int j = 0; j < 4; ++j) full |= (__builtin_bit_cast(u4v, x[kb])[j] & 0x7f807f80u) + 0x00800080u;
    return __builtin_amdgcn_ballot_w64((full & 0x80008000u) != 0) != 0;
}
__device__ __forceinline__ void finite_only(s8 (&x)[2]) {
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[kb][e] = is_special((uint16_t)x[kb][e]) ? (short)0 : x[kb][e];
}
// y, lane = token 16 it + r, entries the 4 channels at `x` (token 0), and M as ChainSmem holds it.
__device__ __forceinline__ void add_special(const uint16_t *m, const uint16_t *x, f4 (&y)[4]) {
    const int r = threadIdx.x & 15;
#pragma unroll 1
    for (int j = 0; j < kL; ++j) {
        const s4 xj = *reinterpret_cast<const s4 *>(x + j * kXPitch);
        bool any = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) any |= is_special((uint16_t)xj[e]);
        if (__builtin_amdgcn_ballot_w64(any) == 0) continue;
        const int jt = j >> 4;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            if (it < jt) continue;
            float mij = 0.f;
#pragma unroll
            for (int part = kParts - 1; part >= 0; --part)
                mij += bf16_bits_to_f32(m[(((4 * part + it) * 2 + (jt >> 1)) * 64 + 16 * ((j & 15) >> 2) + r) * 8 + 4 * (jt & 1) + (j & 3)]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (16 * it + r >= j && is_special((uint16_t)xj[e])) y[it][e] += mij * bf16_bits_to_f32((uint16_t)xj[e]);
        }
    }
}

// kReverse: the chains of the gradient of the state, from the last token to the
// first: D <- e^{G_63} D + sum_i e^{G_i} d_out_i C_i^T.
// With kCausal, a NaN or infinity in x as add_special has it; otherwise returns whether
// that is needed.
template <int kN, int kPass, bool kReverse, bool kCausal>
__device__ __forceinline__ bool walk_piece(const SsmChainArgs &a, ChainSmem<kN, kPass == kOutputs> &sm) {
    constexpr bool kOut = kPass == kOutputs;
    // The states that the gradient reads are kept as accumulators hold them, 16
    // bytes a lane: those of the scan as S (rows: channels), so that a pair of
    // tiles is an operand along channels, those of its gradient as here, S^T.
    constexpr bool kSwapped = kPass == kSave && !kReverse;
    constexpr int kTiles = kN / 16, kQ = kN / 32;
    constexpr int kGroup = kOut ? 4 : 1;  // state tiles updated side by side, as registers allow
    int64_t index, h, pb;
    place(a, index, h, pb);
    const Piece p = piece_of(a, index);
    if (!p.valid) return false;
    if (kPass == kPieces && (kReverse ? p.first : p.last)) return false;  // nothing follows it

    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int64_t grp = h / (a.H / a.G);
    const float nA2 = -decay_rate(a.A_log[h]) * kLog2e;
    const float bias = a.dt_bias ? a.dt_bias[h] : 0.f;
    const float Dh = kOut && a.D ? a.D[h] : 0.f;
    const uint16_t *xrow = a.x + p.row0 * a.xb + p.t0 * a.xt + h * a.P + pb * kPB;
    const uint16_t *krow = a.k + p.row0 * a.kb + p.t0 * a.kt + grp * kN;
    const uint16_t *crow = kOut ? a.c + p.row0 * a.cb + p.t0 * a.ct + grp * kN : nullptr;
    const uint16_t *drow = a.dt + p.row0 * a.dtb + p.t0 * a.dtt + h;
    uint16_t *orow = kOut ? a.out + ((p.row0 * a.T + p.t0) * a.H + h) * a.P + pb * kPB : nullptr;
    // this lane's rows of a state tensor: channel 16 w + r, entries 32 q + 8 g ..
    const int64_t sbase = (h * a.P + pb * kPB + 16 * w + r) * kN + 8 * g;
    const int64_t sseq = p.n * a.H * a.P * kN + sbase, spiece = p.slot * a.H * a.P * kN + sbase;

    const int chunks = (p.count + kL - 1) / kL;
    // where only the states are kept, what leaves the piece is not needed
    const bool leave = kPass == kSave && !(kReverse && p.first && a.ht);
    const int steps = chunks - leave;
    Rows<kN, kThreads> rk, rc;
    Rows<kPB, kThreads> rx;
    rk.init(a.kt, kPitch<kN>);
    if constexpr (kOut) rc.init(a.ct, kPitch<kN>);
    rx.init(a.xt, kXPitch);
    uint32_t rdt = 0;
    // step sizes of the piece's chunk c, as loaded: used, and so waited for, later; tokens
    // behind the last one read it again
    auto raw_dt = [&](int c) -> uint32_t {
        const int t = c * kL + lane;
        return drow[(int64_t)(t < p.count ? t : p.count - 1) * a.dtt];
    };
    // The next chunk's rows, in parts: a dozen loads at once fill the memory pipeline's
    // queue and hold up what follows (at 8192 x 64 heads, 1500 of 8600 cycles a chunk).
    constexpr int kX = 1, kK = 2, kC = 4, kAll = 7;
    auto fetch = [&](int i, const int what) {
        if (i > 0 && i >= steps) return;
        const int c = kReverse ? chunks - 1 - i : i;
        const int rows = p.count - c * kL < kL ? p.count - c * kL : kL;
        const int64_t t = (int64_t)c * kL;
        if (!kOut && w == kStepper) rdt = raw_dt(c);
        if (what & kX) rx.load(xrow + t * a.xt, rows);
        if (what & kK) rk.load(krow + t * a.kt, rows);
        if (kOut && what & kC) rc.load(crow + t * a.ct, rows);
    };
    fetch(0, kAll);

    // ---- the state at the start
    f4 S[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) S[t] = f4{0.f, 0.f, 0.f, 0.f};
    if constexpr (kPass != kPieces) {
        const bool whole = p.first && p.last;  // a single piece starts from the initial state itself
        const void *src = whole ? a.h0 : a.state;
        const int f32 = whole ? a.h0_f32 : 1;
        const int64_t from = whole ? p.n : p.slot;
        if (src) {
            if constexpr (kSwapped) {
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        S[t][e] = load_any(src, ((from * a.H + h) * a.P + pb * kPB + 16 * w + 4 * g + e) * kN + 16 * t + r, f32);
            } else {
#pragma unroll
                for (int q = 0; q < kQ; ++q) {
                    float v[8];
                    load_state8(src, (whole ? sseq : spiece) + 32 * q, f32, v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        S[2 * q][e] = v[e];
                        S[2 * q + 1][e] = v[4 + e];
                    }
                }
            }
        }
    }

    // The outputs of the chunk before: a thread takes them from where it then stores x.
    constexpr int kHalf = kL / 2;  // rows of a pass over x
    uint4 out0, out1;
    const uint32_t orow_step = (uint32_t)(a.H * a.P);
    const uint32_t ooff = (uint32_t)(threadIdx.x >> 3) * orow_step + 8 * (threadIdx.x & 7);
    uint16_t *const oplace = sm.x + (threadIdx.x >> 3) * kXPitch + 8 * (threadIdx.x & 7);
    auto take = [&] {
        out0 = *reinterpret_cast<const uint4 *>(oplace);
        out1 = *reinterpret_cast<const uint4 *>(oplace + kHalf * kXPitch);
    };
    auto put = [&](int rows) {
        const int t = threadIdx.x >> 3;
        if (t < rows) *reinterpret_cast<uint4 *>(orow + ooff) = out0;
        if (kHalf + t < rows) *reinterpret_cast<uint4 *>(orow + ooff + kHalf * orow_step) = out1;
        orow += (int64_t)kL * orow_step;
    };
    // this wave's tiles of M left of the diagonal: rows 1 and 2 of column 0; (2, 1) and
    // (3, 0); rows 3 of columns 1 and 2
    const int it0 = w == 0 ? 1 : w == 1 ? 2 : 3, jt0 = w == 0 ? 0 : 1, it1 = w == 0 ? 2 : 3, jt1 = w == 2 ? 2 : 0;
    float total = 0.f;
    [[maybe_unused]] bool seen = false;
    if (kOut && threadIdx.x == 0) sm.special = 0;
    // Outputs: the next chunk's step sizes are taken beside this one's M, by a wave
    // with few of its tiles.
    if (kOut && w == kStepper) {
        step_sizes(bf16_bits_to_f32(raw_dt(0)), lane < p.count, bias, nA2, sm.s[0]);
        tile_decays(sm.s[0], sm.t[0]);
        rdt = raw_dt(1);
    }
    if (kOut && w < 2) {  // M's tiles (0, 1) and (2, 3) are zero: half an operand each, all parts
#pragma unroll
        for (int part = 0; part < kParts; ++part)
            *reinterpret_cast<s4 *>(&sm.m[(((4 * part + 2 * w) * 2 + w) * 64 + lane) * 8 + 4]) = s4{0, 0, 0, 0};
    }
    auto keep_state = [&](int c) {
        if (p.chunk0 + c >= a.chunks) return;
        f4 *dst = reinterpret_cast<f4 *>(a.save) +
                  (((p.chunk0 + c) * a.H + h) * (a.P / kPB) + pb) * (kPB * kN / 4) + w * kTiles * 64 + lane;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) dst[t * 64] = S[t];
    };
    // Barriers here order LDS traffic only: the next chunk's loads stay in flight.
    for (int i = 0; i < steps; ++i) {
        const int c = kReverse ? chunks - 1 - i : i;
        const int rows = p.count - c * kL < kL ? p.count - c * kL : kL;
        if (i) lds_barrier();                    // the chunk before is done with
        if (!kOut && w == kStepper) step_sizes(bf16_bits_to_f32(rdt), lane < rows, bias, nA2, sm.s[i & 1]);
        if constexpr (kOut) {
            if (i) take();
        }
        rx.store(sm.x, kXPitch);
        rk.store(sm.k, kPitch<kN>);
        if constexpr (kOut) rc.store(sm.c, kPitch<kN>);
        lds_barrier();
        // What goes to memory goes out here, behind the wait for this chunk's loads and
        // before the next one's: the next wait, which counts both, comes a chunk later.
        if constexpr (kPass == kSave) keep_state(c);
        if constexpr (kOut) {
            if (i > 0) put(kL);
        }
        fetch(i + 1, kOut ? kX : kAll);
        const Steps &st = sm.s[i & 1];
        [[maybe_unused]] const TileDecays &td = sm.t[kOut ? i & 1 : 0];
        const float gl = st.g[kL - 1];

        // x along tokens, for this wave's channels
        s8 xf[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const uint16_t *q = sm.x + (32 * kb + 4 * g + (r >> 2)) * kXPitch + 16 * w + 4 * (r & 3);
            xf[kb] = join(read_tr(q), read_tr(q + 16 * kXPitch));
        }

        f4 y[4];
        if constexpr (kOut) {
            // ---- M, 16 x 16 tiles as B C^T: lane = row i, its entries 4 columns j, half of an
            // operand.  Tiles left of the diagonal take their decays as a product
            // around the tile's first row; the diagonal tiles take the exponentials
            // themselves.  Each wave has a diagonal tile; two of the others go to each wave
            // that takes no step sizes.
            auto scores = [&](const int it, const int jt) {
                f4 cb = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < kQ; ++q)
                    cb = mfma16x16x32_bf16(lds8(sm.k + (16 * jt + r) * kPitch<kN> + 32 * q + 8 * g),
                                           lds8(sm.c + (16 * it + r) * kPitch<kN> + 32 * q + 8 * g), cb);
                return cb;
            };
            auto keep = [&](const int it, const int jt, f4 m) {
                float v[4] = {m[0], m[1], m[2], m[3]};
                keep_parts(v, &sm.m[((it * 2 + (jt >> 1)) * 64 + lane) * 8 + 4 * (jt & 1)], 4 * 2 * 64 * 8);
            };
            auto left = [&](const int it, const int jt, f4 cb) {
                const float upto = td.upto[16 * it + r];
                const f4 b = *reinterpret_cast<const f4 *>(&td.before[it - 1][16 * jt + 4 * g]);
#pragma unroll
                for (int e = 0; e < 4; ++e) cb[e] *= upto * b[e];
                keep(it, jt, cb);
            };
            auto diagonal = [&](f4 cb) {
                const float gi = st.g[16 * w + r], gir = st.gr[16 * w + r];
                const f4 gj = *reinterpret_cast<const f4 *>(&st.g[16 * w + 4 * g]);
                const f4 gjr = *reinterpret_cast<const f4 *>(&st.gr[16 * w + 4 * g]);
                const f4 dj = *reinterpret_cast<const f4 *>(&st.dt[16 * w + 4 * g]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = 4 * g + e;
                    const float v = cb[e] * (__builtin_amdgcn_exp2f((gi - gj[e]) + (gir - gjr[e])) * dj[e]);
                    cb[e] = j < r ? v : j == r ? v + Dh : 0.f;
                }
                keep(w, w, cb);
            };
            if (w == kStepper) {
                const f4 d = scores(w, w);
                if (i + 1 < chunks) {
                    Steps &next = sm.s[(i + 1) & 1];
                    step_sizes(bf16_bits_to_f32(rdt), lane < p.count - (i + 1) * kL, bias, nA2, next);
                    tile_decays(next, sm.t[(i + 1) & 1]);
                }
                rdt = raw_dt(i + 2);
                diagonal(d);
            } else {
                const f4 d = scores(w, w), l0 = scores(it0, jt0), l1 = scores(it1, jt1);
                left(it0, jt0, l0);
                left(it1, jt1, l1);
                diagonal(d);
            }
            fetch(i + 1, kK);
            // ---- outputs from the entering state, transposed: lane = token, entries 4
            // neighbouring channels
#pragma unroll
            for (int it = 0; it < 4; ++it) y[it] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = S[2 * q][e];
                    v[4 + e] = S[2 * q + 1][e];
                }
                s8 sv[kParts];
                split3(v, sv[0], sv[1], sv[2]);
                // products into one accumulator are four apart: none waits for the one before
                s8 cv[4];
#pragma unroll
                for (int it = 0; it < 4; ++it) cv[it] = lds8(sm.c + (16 * it + r) * kPitch<kN> + 32 * q + 8 * g);
#pragma unroll
                for (int part = 0; part < kParts; ++part)
#pragma unroll
                    for (int it = 0; it < 4; ++it) y[it] = mfma16x16x32_bf16(sv[part], cv[it], y[it]);
            }
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const float d = st.from[16 * it + r];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[it][e] *= d;
            }
        }

        // ---- the state at the chunk's end
        const float dl = __builtin_amdgcn_exp2f(gl);
        total += gl;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[t][e] *= dl;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            float v[8];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float *wp = kReverse ? st.from : st.w;
                const float4 wj = *reinterpret_cast<const float4 *>(wp + 32 * kb + 16 * half + 4 * g);
                const float wv[4] = {wj.x, wj.y, wj.z, wj.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * half + e] = wv[e] * bf16_bits_to_f32((uint16_t)xf[kb][4 * half + e]);
            }
            s8 xs[kParts];
            split3(v, xs[0], xs[1], xs[2]);
#pragma unroll
            for (int t0 = 0; t0 < kTiles; t0 += kGroup) {
                s8 kv[kGroup];
#pragma unroll
                for (int t = t0; t < t0 + kGroup; ++t) {
                    const int col = kSwapped ? 16 * t + 4 * (r & 3) : 32 * (t >> 1) + 8 * (r & 3) + 4 * (t & 1);
                    const uint16_t *q = sm.k + (32 * kb + 4 * g + (r >> 2)) * kPitch<kN> + col;
                    kv[t - t0] = join(read_tr(q), read_tr(q + 16 * kPitch<kN>));
                }
#pragma unroll
                for (int part = 0; part < kParts; ++part)
#pragma unroll
                    for (int t = t0; t < t0 + kGroup; ++t)
                        S[t] = kSwapped ? mfma16x16x32_bf16(xs[part], kv[t - t0], S[t]) : mfma16x16x32_bf16(kv[t - t0], xs[part], S[t]);
            }
        }
        // ---- outputs from the chunk's own tokens
        if constexpr (kOut) {
            fetch(i + 1, kC);
            const bool special = kCausal && any_special(xf);
            if (special) finite_only(xf);
            lds_barrier();
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int part = 0; part < kParts; ++part)
#pragma unroll
                    for (int it = 2 * kb; it < 4; ++it)
                        y[it] = mfma16x16x32_bf16(xf[kb], lds8(&sm.m[(((4 * part + it) * 2 + kb) * 64 + lane) * 8]), y[it]);
            if (special) add_special(sm.m, sm.x + 16 * w + 4 * g, y);
#pragma unroll
            for (int e = 0; e < 4; ++e) seen |= !kCausal && !__builtin_isfinite(y[3][e]);
#pragma unroll
            for (int it = 0; it < 4; ++it)
                *reinterpret_cast<uint2 *>(sm.x + (16 * it + r) * kXPitch + 16 * w + 4 * g) =
                    make_uint2(pack_pair(y[it][0], y[it][1]), pack_pair(y[it][2], y[it][3]));
        }
    }
    if constexpr (kOut) {
        if (seen) sm.special = 1;
        lds_barrier();
        if (!kCausal && __builtin_amdgcn_readfirstlane(sm.special)) {
            lds_barrier();
            return true;
        }
        take();
        put(p.count - (chunks - 1) * kL);
    }

    if constexpr (kPass == kSave) {
        if (leave) keep_state(kReverse ? 0 : chunks - 1);
    }

    // ---- the state at the end
    void *dst = kPass == kPieces ? a.state : kSwapped ? nullptr : (kReverse ? p.first : p.last) ? a.ht : nullptr;
    if (dst) {
#pragma unroll
        for (int q = 0; q < kQ; ++q)
            store_state8(dst, (kPass == kPieces ? spiece : sseq) + 32 * q, kPass == kPieces ? 1 : a.ht_f32, S[2 * q], S[2 * q + 1]);
    }
    if (kPass == kPieces && threadIdx.x == 0 && pb == 0) a.decay[p.slot * a.H + h] = total;
    return false;
}

template <int kN, int kPass, bool kReverse>
__global__ __launch_bounds__(kThreads, kPass == kOutputs ? 2 : 4) void kda_ssm_chain_kernel(SsmChainArgs a) {
    __shared__ ChainSmem<kN, kPass == kOutputs> sm;
    const bool again = walk_piece<kN, kPass, kReverse, false>(a, sm);
    if constexpr (kPass == kOutputs) {
        if (again) {
            // the arguments are read anew: kept over the first walk, they would take its registers
            auto p = (const __attribute__((address_space(4))) SsmChainArgs *)__builtin_amdgcn_kernarg_segment_ptr();
            asm volatile("" : "+s"(p));
            const SsmChainArgs b = *(const SsmChainArgs *)p;
            walk_piece<kN, kPass, kReverse, true>(b, sm);
        }
    }
}

// The states entering the pieces of every sequence with several of them, in
// place of the pieces' own states: E_0 = h0, E_{k+1} = 2^decay_k E_k + own_k (last
// to first when reversed).  Sequences without tokens get their final state here.
// One thread per 4 entries of a head's state; the loads of kBatch pieces are in
// flight together, and the next ones' while they are added up.
constexpr int kBatch = 8;
template <bool k> struct Flag { static constexpr bool value = k; };

template <int kN, bool kReverse>
__global__ __launch_bounds__(kThreads) void kda_ssm_scan_kernel(SsmChainArgs a) {
    const int64_t size = a.P * kN;
    const int64_t per = size / (4 * kThreads);
    for (int64_t u = blockIdx.x; u < a.seqs * a.H * per; u += gridDim.x) {
        const int64_t part = u % per, nh = u / per;
        const int64_t n = nh / a.H, h = nh - n * a.H;
        const int64_t off = part * 4 * kThreads + threadIdx.x * 4;
        int64_t first, count, pieces;
        if (a.cu) {
            first = a.slot_off[n];
            count = a.slot_off[n + 1] - first;
            pieces = a.piece_off[n + 1] - a.piece_off[n];
        } else {
            first = n * a.pps;
            count = pieces = a.pps;
        }
        if (pieces > 0 && count < 2) continue;
        f4 E = {0.f, 0.f, 0.f, 0.f};
        if (a.h0)
#pragma unroll
            for (int e = 0; e < 4; ++e) E[e] = load_any(a.h0, nh * size + off + e, a.h0_f32);
        if (pieces == 0) {
            if (a.ht)
#pragma unroll
                for (int e = 0; e < 4; ++e) store_any(a.ht, nh * size + off + e, a.ht_f32, E[e]);
            continue;
        }
        f4 *state = reinterpret_cast<f4 *>(a.state + h * size + off);
        const int64_t step = a.H * size / 4;
        auto piece = [&](int64_t i) { return first + (kReverse ? count - 1 - i : i); };
        // Many pieces: no branches around the loads, and the last place read again behind the
        // last one; few: no loads that nothing takes (nothing takes the last one's state).
        auto load = [&](int64_t i0, f4 (&own)[kBatch], float (&d)[kBatch], auto many) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int64_t k = piece(i0 + i < count ? i0 + i : count - 1);
                if (!decltype(many)::value && i0 + i + 1 >= count) break;
                own[i] = state[k * step];
                d[i] = a.decay[k * a.H + h];
            }
        };
        auto walk = [&](int64_t i0, const f4 (&own)[kBatch], const float (&d)[kBatch], int n) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (i >= n) break;
                state[piece(i0 + i) * step] = E;
                const float m = __builtin_amdgcn_exp2f(d[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) E[e] = m * E[e] + own[i][e];
            }
        };
        f4 own0[kBatch], own1[kBatch];
        float d0[kBatch], d1[kBatch];
        int64_t i0 = 0;
        if (count < 2 * kBatch) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                own0[i] = f4{0.f, 0.f, 0.f, 0.f};
                d0[i] = 0.f;
            }
            for (; i0 < count; i0 += kBatch) {
                load(i0, own0, d0, Flag<false>{});
                walk(i0, own0, d0, (int)(count - i0));
            }
            continue;
        }
        load(0, own0, d0, Flag<true>{});
        for (; i0 + 2 * kBatch <= count; i0 += 2 * kBatch) {
            load(i0 + kBatch, own1, d1, Flag<true>{});
            walk(i0, own0, d0, kBatch);
            load(i0 + 2 * kBatch, own0, d0, Flag<true>{});
            walk(i0 + kBatch, own1, d1, kBatch);
        }
        const int left = (int)(count - i0);      // below 2 kBatch, the first of them loaded
        if (left > kBatch) load(i0 + kBatch, own1, d1, Flag<true>{});
        walk(i0, own0, d0, left);
        if (left > kBatch) walk(i0 + kBatch, own1, d1, left - kBatch);
    }
}

// First piece, chunk and slot of every sequence of a packed batch: running sums
// over the sequences by one workgroup.  Lengths that overlap (which no batch
// has) could add up to more than the workspace holds: the tables end there.
__global__ __launch_bounds__(1024) void kda_ssm_table_kernel(SsmTables a) {
    __shared__ int64_t sum[3][1024];
    int32_t *const tables[3] = {a.piece_off, a.chunk_off, a.slot_off};
    const int64_t most[3] = {a.pieces, a.chunks, a.slots};
    const int tid = threadIdx.x;
    int64_t before[3] = {0, 0, 0};
    for (int64_t base = 0; base < a.seqs; base += 1024) {
        const int64_t n = base + tid;
        int64_t own[3] = {0, 0, 0};
        if (n < a.seqs) {
            const int64_t len = clamp_to(a.cu[n + 1], a.T) - clamp_to(a.cu[n], a.T);
            own[1] = len > 0 ? (len + kL - 1) / kL : 0;
            own[0] = (own[1] + a.pc - 1) / a.pc;
            own[2] = own[0] > 1 ? own[0] : 0;
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) sum[k][tid] = own[k];
        __syncthreads();
        for (int d = 1; d < 1024; d <<= 1) {
            int64_t v[3];
#pragma unroll
            for (int k = 0; k < 3; ++k) v[k] = tid >= d ? sum[k][tid - d] : 0;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 3; ++k) sum[k][tid] += v[k];
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (n < a.seqs) tables[k][n] = (int32_t)clamp_to(before[k] + sum[k][tid] - own[k], most[k]);
            before[k] += sum[k][1023];
        }
        __syncthreads();
    }
    if (tid == 0)
#pragma unroll
        for (int k = 0; k < 3; ++k) tables[k][a.seqs] = (int32_t)clamp_to(before[k], most[k]);
}

template <int kN, int kPass, bool kReverse>
hipError_t launch(const SsmChainArgs &a, hipStream_t s) {
    SsmChainArgs b = a;
    return launch_groups(grid_size(a), a.launch_cap, [&](int64_t base, dim3 grid) {
        b.base = base;
        hipLaunchKernelGGL((kda_ssm_chain_kernel<kN, kPass, kReverse>), grid, dim3(kThreads), 0, s, b);
    });
}

}  // namespace

hipError_t kda_launch_ssm_table(const SsmTables &a, hipStream_t s) {
    hipLaunchKernelGGL(kda_ssm_table_kernel, dim3(1), dim3(1024), 0, s, a);
    return hipGetLastError();
}

hipError_t kda_launch_ssm_pieces(const SsmChainArgs &a, int N, bool reverse, hipStream_t s) {
    if (N == 128) return reverse ? launch<128, kPieces, true>(a, s) : launch<128, kPieces, false>(a, s);
    return reverse ? launch<64, kPieces, true>(a, s) : launch<64, kPieces, false>(a, s);
}

hipError_t kda_launch_ssm_scan(const SsmChainArgs &a, int N, bool reverse, hipStream_t s) {
    const int64_t units = a.seqs * a.H * (a.P * N / (4 * kThreads));
    const unsigned grid = (unsigned)(units < (1 << 16) ? units : (1 << 16));
    if (N == 128) {
        if (reverse) hipLaunchKernelGGL((kda_ssm_scan_kernel<128, true>), dim3(grid), dim3(kThreads), 0, s, a);
        else hipLaunchKernelGGL((kda_ssm_scan_kernel<128, false>), dim3(grid), dim3(kThreads), 0, s, a);
    } else {
        if (reverse) hipLaunchKernelGGL((kda_ssm_scan_kernel<64, true>), dim3(grid), dim3(kThreads), 0, s, a);
        else hipLaunchKernelGGL((kda_ssm_scan_kernel<64, false>), dim3(grid), dim3(kThreads), 0, s, a);
    }
    return hipGetLastError();
}

hipError_t kda_launch_ssm_save(const SsmChainArgs &a, int N, bool reverse, hipStream_t s) {
    if (N == 128) return reverse ? launch<128, kSave, true>(a, s) : launch<128, kSave, false>(a, s);
    return reverse ? launch<64, kSave, true>(a, s) : launch<64, kSave, false>(a, s);
}

hipError_t kda_launch_ssm_chain(const SsmChainArgs &a, int N, hipStream_t s) {
    return N == 128 ? launch<128, kOutputs, false>(a, s) : launch<64, kOutputs, false>(a, s);
}
