// kda_layer_args.h -- kernel arguments and launchers of the layer operators
// (include/kda_layer.h): RMS normalisation, short convolution, state-space scan.
#pragma once
#include "kda_common.h"

namespace kda {

struct NormArgs {
    const uint16_t *x;         // bf16 rows, xs elements apart
    const void *res;           // residual rows (bf16 or fp32), rs elements apart, or nullptr
    const void *w;             // [D]
    void *res_out;             // contiguous, of the residual's type, or nullptr
    void *out;                 // bf16 or e4m3, contiguous
    float *scales;             // quantised output: [rows, ceil(D / group)] or [rows, 1]
    int64_t rows, D, xs, rs;
    int64_t groups;            // scales per row
    float eps;
    int res_f32, w_f32;
    int quant;                 // 0: bf16, 1: e4m3 with one scale per row, 2: one per 128 columns
};

struct NormBwdArgs {
    const void *h;             // bf16 or fp32 rows, hs elements apart
    const void *w;
    const uint16_t *dy;        // rows ds elements apart
    const void *dres;          // of h's type, rows rs elements apart, or nullptr
    uint16_t *dx;
    float *dresidual;          // or nullptr
    float *dw;
    float *part;               // [parts, D] partial sums of dw
    float *rstd;               // [rows] (the scalar path)
    int64_t rows, D, hs, ds, rs;
    int64_t parts;
    float eps;
    int h_f32, w_f32;
};

// Packed batches: cu with the lengths; otherwise sequence n is batch row n of T tokens.
struct ConvArgs {
    const uint16_t *x;
    const void *w, *bias;      // [D, W], [D] or nullptr
    const void *h0;            // [N, W - 1, D] or nullptr
    void *ht;
    const int64_t *cu;
    uint16_t *out;
    int64_t B, T, D, N, xb, xt;
    int silu, w_f32, h0_f32, ht_f32;
    // gradient
    const uint16_t *dy;
    int64_t db_, dt_;          // strides of dy
    const void *dht;           // of ht's type, or nullptr
    uint16_t *dx;
    float *dw, *dbias, *dh0;
    float *part;               // [parts, W + 1, D] partial sums of dw and dbias
    int64_t parts;
};

struct SsmArgs {
    const uint16_t *x, *dt, *Bm, *Cm;
    const float *A_log, *dt_bias, *D;
    const void *h0;
    void *ht;
    const int64_t *cu;
    uint16_t *out;
    int64_t B, T, H, P, G, N, num_seqs;
    int64_t xb, xt, dtb, dtt, bb, bt, cb, ct;
    int h0_f32, ht_f32;
    int64_t launch_cap;        // kda_ssm_desc_t::launch_piece
};

// The scan's state chains.  A piece is up to `pc` 64-token chunks of one
// sequence, walked through in order by one workgroup per (head, 64 channels).
// The tables of a packed batch give the first piece and the first chunk of
// every sequence, and the first slot for a piece's state, which only the pieces of
// sequences with several have; otherwise every sequence has `pps` pieces and `cps`
// chunks, and the slots are the pieces.
struct SsmChainArgs {
    const uint16_t *x;         // [tokens, H, P]: x, or d_out backwards
    const uint16_t *k;         // [tokens, G, N]: B, or C backwards
    const uint16_t *c;         // C (outputs only)
    const uint16_t *dt;
    int64_t xb, xt, kb, kt, cb, ct, dtb, dtt;
    const float *A_log, *dt_bias, *D;
    const int64_t *cu;
    const int32_t *piece_off, *chunk_off, *slot_off;
    int64_t T, H, P, G, seqs;
    int64_t pieces, chunks, slots;  // of the batch (upper bounds when packed)
    int64_t pps, cps;
    int pc;
    const void *h0;            // state at the chains' start, or nullptr
    void *ht;                  // state at their end, or nullptr
    int h0_f32, ht_f32;
    float *state;              // [slots, H, P, N]: a piece's own state, then the one entering it
    float *decay;              // [slots, H]: log2 of a piece's decay
    float *save;               // [chunks, H, P / 64, 64 N]: state entering every chunk (kda_ssm.hip)
    uint16_t *out;
    int64_t launch_cap, base;  // base: first workgroup of this launch; set by the launcher
};

// The scan's gradient, chunk by chunk, from the states entering every chunk
// (hs) and the gradients of those leaving it (ds).
struct SsmGradArgs {
    const uint16_t *x, *Bm, *Cm, *dt, *dy;
    int64_t xb, xt, bb, bt, cb, ct, dtb, dtt, yb, yt;
    const float *A_log, *dt_bias, *D;
    const int64_t *cu;
    const int32_t *chunk_off;
    int64_t T, H, P, G, seqs;
    int64_t chunks, cps;
    int share;                 // heads of a group per workgroup
    int shares;                // workgroups per chunk and group
    const float *hs, *ds;
    uint16_t *dx, *ddt, *dB, *dC;
    float *part;               // [2][shares][chunks][G][64][N]: dB, dC (with more than one share)
    float *psum;               // [chunks][H][4]: the parameters' gradients
    float *dA_log, *ddt_bias, *dD;
    int64_t launch_cap, base;
};

// Launches of at most 2^23 workgroups (or `cap` of them, kda_ssm_desc_t::launch_piece),
// since a launch's work-items are counted in 32 bits: calls launch(first workgroup,
// number) for every one of them.  Their size is a multiple of 8, which keeps the XCD of
// every workgroup.
template <typename F>
inline hipError_t launch_groups(int64_t groups, int64_t cap, F launch) {
    const int64_t most = (launch_piece(int64_t(1) << 23, cap) + 7) / 8 * 8;
    for (int64_t base = 0; base < groups; base += most) {
        launch(base, dim3((unsigned)(groups - base < most ? groups - base : most)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// fp32 -> two bf16 in one word (round to nearest even), low half first.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return (uint32_t)f32_to_bf16_bits(lo) | ((uint32_t)f32_to_bf16_bits(hi) << 16);
}

// A parameter or state entry of either type.
__device__ __forceinline__ float load_any(const void *p, int64_t i, int f32) {
    return f32 ? reinterpret_cast<const float *>(p)[i] : bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(p)[i]);
}
__device__ __forceinline__ void store_any(void *p, int64_t i, int f32, float v) {
    if (f32) reinterpret_cast<float *>(p)[i] = v;
    else reinterpret_cast<uint16_t *>(p)[i] = f32_to_bf16_bits(v);
}

// e^x with the rounding of x log2(e) made good: the hardware's exp2 of the rounded
// product alone is off by |x| 2^-24, relative, which a step size of e^-7 would show.
__device__ __forceinline__ float exact_exp(float x) {
    constexpr float kHi = 1.44269502f, kLo = 1.92596303e-8f;  // log2(e) = kHi + kLo
    const float p = x * kHi;
    const float rest = __builtin_fmaf(x, kHi, -p) + x * kLo;
    const float e = __builtin_amdgcn_exp2f(p);
    return fabsf(p) < 200.0f ? __builtin_fmaf(e, rest * 0.693147182f, e) : e;  // beyond: 0 or infinity
}

// The scan's decay rate e^A_log, at most 2^100, so that its products with step sizes (up
// to 2^20) and their sums over a chunk stay finite, and zero without a step: rates like
// that leave nothing of a state, whatever the step.
__device__ __forceinline__ float decay_rate(float A_log) {
    const float e = exact_exp(A_log);
    return e > 0x1p100f ? 0x1p100f : e;          // false for NaN
}

// softplus(x) = max(x, 0) + log1p(t), t = e^-|x| <= 1, to about 2^-23 relative:
// log1p(t) = 2 atanh(z) with z = t / (2 + t) <= 1/3, by the series to z^15 (the next
// term is below 2^-27 relative).
__device__ __forceinline__ float softplus(float x) {
    const float t = exact_exp(-fabsf(x));
    const float z = t * fast_rcp(2.0f + t), q = z * z;
    float s = 1.0f / 15.0f;
    s = __builtin_fmaf(s, q, 1.0f / 13.0f);
    s = __builtin_fmaf(s, q, 1.0f / 11.0f);
    s = __builtin_fmaf(s, q, 1.0f / 9.0f);
    s = __builtin_fmaf(s, q, 1.0f / 7.0f);
    s = __builtin_fmaf(s, q, 1.0f / 5.0f);
    s = __builtin_fmaf(s, q, 1.0f / 3.0f);
    const float l = 2.0f * __builtin_fmaf(z * q, s, z);
    return fmaxf(x, 0.0f) + l;
}
__device__ __forceinline__ float sigmoid(float x) { return fast_rcp(1.0f + fast_exp(-x)); }

}  // namespace kda

hipError_t kda_launch_rmsnorm(const kda::NormArgs &a, hipStream_t s);
// Partial dweight rows the gradient writes for these shapes.
int64_t kda_rmsnorm_parts(int64_t rows, int64_t D);
hipError_t kda_launch_rmsnorm_bwd(const kda::NormBwdArgs &a, hipStream_t s);
hipError_t kda_launch_conv(const kda::ConvArgs &a, int W, hipStream_t s);
hipError_t kda_launch_conv_decode(const kda::ConvArgs &a, int W, hipStream_t s);
int64_t kda_conv_parts(int64_t B, int64_t T, int64_t D);
hipError_t kda_launch_conv_bwd(const kda::ConvArgs &a, int W, hipStream_t s);
hipError_t kda_launch_ssm_decode(const kda::SsmArgs &a, hipStream_t s);
// The tables of a packed batch (SsmChainArgs), [seqs + 1] each; its pieces, chunks and
// slots are the most that they may count.
struct SsmTables {
    const int64_t *cu;
    int64_t seqs, T;
    int pc;
    int64_t pieces, chunks, slots;
    int32_t *piece_off, *chunk_off, *slot_off;
};
hipError_t kda_launch_ssm_table(const SsmTables &a, hipStream_t s);
// The pieces' own states, from zero (all but a sequence's last piece in walking order).
hipError_t kda_launch_ssm_pieces(const kda::SsmChainArgs &a, int N, bool reverse, hipStream_t s);
// The state entering every piece from the pieces' own ones, and the final
// states of sequences without tokens.
hipError_t kda_launch_ssm_scan(const kda::SsmChainArgs &a, int N, bool reverse, hipStream_t s);
// The chains from the entering states, keeping the state entering every chunk
// (and, reversed, giving the initial state's gradient).
hipError_t kda_launch_ssm_save(const kda::SsmChainArgs &a, int N, bool reverse, hipStream_t s);
hipError_t kda_launch_ssm_grad(const kda::SsmGradArgs &a, int N, hipStream_t s);
// The chains from the entering states: outputs and final states.
hipError_t kda_launch_ssm_chain(const kda::SsmChainArgs &a, int N, hipStream_t s);
