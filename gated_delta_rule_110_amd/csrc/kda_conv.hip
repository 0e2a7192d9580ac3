// kda_conv.hip -- the short causal depthwise convolution (gfx950): prompts,
// one token per sequence, and the gradient.
//
//   pre_t = bias + sum_k w_k x_{t - (W - 1) + k},   out_t = pre_t or silu(pre_t)
//
// per channel, the W - 1 inputs before a sequence's first token coming from its
// state.  Two operations per loaded value and tap: bound by memory traffic (x
// once, out once).  A lane holds 4 neighbouring channels (8 bytes per token and
// access, 512 per wave) and walks over a run of tokens with the last W - 1
// inputs in registers, so that x is read once plus W - 1 rows per run.  Where the
// channel count or a stride is no multiple of 8, or an address none of 16 bytes, the
// same code runs with one channel per lane.  Measured: 4 x 2048 tokens of 12288 channels
// 84 us, 32768 packed tokens of 4352 112 us (4.8 and 5.1 TB/s of what has to be read
// and written; the runtime's copy reaches 5.1, an elementwise one of a GiB 6.2), the
// gradient of 8192 x 4352 47 us and 5 for the weights' sum (4.1 TB/s: each run reads
// W - 1 tokens of its neighbour's again), one token of 64 sequences of 12288 5 us, all
// of it latency.
#include "kda_layer_args.h"

using namespace kda;

namespace {

constexpr int kLanes = 64;       // channel groups per workgroup (one wave wide)
constexpr int kWaves = 4;        // token runs per workgroup
constexpr int kRun = 16;         // tokens per run, forward: their loads are all in flight together
constexpr int kBwdRun = 32;      // tokens per run, gradient
constexpr int64_t kMaxGridY = 65535;

// kC neighbouring bf16 values as loaded, until they are used.
template <int kC> struct Raw;
template <> struct Raw<4> {
    uint2 v;
    __device__ __forceinline__ void load(const uint16_t *p) { v = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void get(float *o) const {
        o[0] = __uint_as_float(v.x << 16); o[1] = __uint_as_float(v.x & 0xffff0000u);
        o[2] = __uint_as_float(v.y << 16); o[3] = __uint_as_float(v.y & 0xffff0000u);
    }
};
template <> struct Raw<1> {
    uint16_t v;
    __device__ __forceinline__ void load(const uint16_t *p) { v = *p; }
    __device__ __forceinline__ void get(float *o) const { o[0] = bf16_bits_to_f32(v); }
};
template <int kC>
__device__ __forceinline__ void load_c(const uint16_t *p, float *o) {
    Raw<kC> r;
    r.load(p);
    r.get(o);
}
template <int kC>
__device__ __forceinline__ void store_c(uint16_t *p, const float *v) {
    if constexpr (kC == 4) *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    else *p = f32_to_bf16_bits(v[0]);
}
// kC entries of a state or parameter row of either type.
template <int kC>
__device__ __forceinline__ void load_any_c(const void *p, int64_t i, int f32, float *o) {
    if constexpr (kC == 1) {
        o[0] = load_any(p, i, f32);
    } else if (f32) {
#pragma unroll
        for (int j = 0; j < kC; j += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p) + i + j);
            o[j] = a.x; o[j + 1] = a.y; o[j + 2] = a.z; o[j + 3] = a.w;
        }
    } else {
        load_c<kC>(reinterpret_cast<const uint16_t *>(p) + i, o);
    }
}
template <int kC>
__device__ __forceinline__ void store_f32_c(float *p, const float *v) {
    if constexpr (kC == 1) p[0] = v[0];
    else {
#pragma unroll
        for (int j = 0; j < kC; j += 4) *reinterpret_cast<float4 *>(p + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
}
template <int kC>
__device__ __forceinline__ void store_any_c(void *p, int64_t i, int f32, const float *v) {
    if (f32) store_f32_c<kC>(reinterpret_cast<float *>(p) + i, v);
    else store_c<kC>(reinterpret_cast<uint16_t *>(p) + i, v);
}

// The lane's filter: w[k][e] for channel c + e.  With several channels its kC kW
// entries are one aligned piece.
template <int kC, int kW>
__device__ __forceinline__ void load_filter(const ConvArgs &a, int64_t c, float (&w)[kW][kC], float (&b)[kC]) {
    float f[kW * kC];
#pragma unroll
    for (int i = 0; i < kW; ++i) load_any_c<kC>(a.w, c * kW + i * kC, a.w_f32, &f[i * kC]);
#pragma unroll
    for (int e = 0; e < kC; ++e) {
        b[e] = 0.f;
#pragma unroll
        for (int k = 0; k < kW; ++k) w[k][e] = f[e * kW + k];
    }
    if (a.bias) load_any_c<kC>(a.bias, c, a.w_f32, b);
}

// Sequences of a batch: their first token and the one behind their last, in
// the flat order b T + t.  Lengths are clamped to the batch's tokens.
struct Seqs {
    const int64_t *cu;
    int64_t T, N, total;
    __device__ __forceinline__ int64_t begin(int64_t n) const { return cu ? clamp(cu[n]) : n * T; }
    __device__ __forceinline__ int64_t end(int64_t n) const { return cu ? clamp(cu[n + 1]) : (n + 1) * T; }
    __device__ __forceinline__ int64_t clamp(int64_t v) const { return v < 0 ? 0 : v > total ? total : v; }
    // The sequence that holds token t, or N if none does (t behind the last):
    // the first n with end(n) > t, by halving.
    __device__ __forceinline__ int64_t of(int64_t t) const {
        if (!cu) return t / T;
        int64_t lo = 0, hi = N;
        while (lo < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if (cu[mid + 1] > t) hi = mid; else lo = mid + 1;
        }
        return lo;
    }
};
__device__ __forceinline__ Seqs seqs_of(const ConvArgs &a) { return Seqs{a.cu, a.T, a.N, a.B * a.T}; }

// Row of x (or dy) of the flat token t.
__device__ __forceinline__ int64_t row_of(int64_t t, int64_t T, int64_t sb, int64_t st) {
    const int64_t b = t / T;
    return b * sb + (t - b * T) * st;
}

// Input number pos (may be negative: from the state) of sequence n.
template <int kC, int kW>
__device__ __forceinline__ void input_at(const ConvArgs &a, int64_t n, int64_t begin, int64_t pos, int64_t c, float *o) {
    if (pos >= 0) {
        load_c<kC>(a.x + row_of(begin + pos, a.T, a.xb, a.xt) + c, o);
    } else if (a.h0 && pos >= -(kW - 1)) {
        load_any_c<kC>(a.h0, (n * (kW - 1) + (kW - 1) + pos) * a.D + c, a.h0_f32, o);
    } else {
#pragma unroll
        for (int e = 0; e < kC; ++e) o[e] = 0.f;
    }
}

template <int kC, int kW>
__device__ __forceinline__ void convolve(const float (&w)[kW][kC], const float (&b)[kC], const float (&win)[kW][kC],
                                         float *pre) {
#pragma unroll
    for (int e = 0; e < kC; ++e) {
        float p = b[e];
#pragma unroll
        for (int k = 0; k < kW; ++k) p += w[k][e] * win[k][e];
        pre[e] = p;
    }
}

// A wave's run of tokens: within one batch row (of T tokens, the packed batch
// being one row), so that its rows are one stride apart.
struct Run {
    int64_t b, t0, stop;      // batch row; flat tokens t0 .. stop - 1
};
__device__ __forceinline__ Run run_of(int64_t u, int64_t runs, int64_t T, int len) {
    Run r;
    r.b = u / runs;
    r.t0 = r.b * T + (u - r.b * runs) * len;
    r.stop = r.t0 + len < (r.b + 1) * T ? r.t0 + len : (r.b + 1) * T;
    return r;
}

template <int kC, int kW>
__device__ __forceinline__ void conv_token(const float (&w)[kW][kC], const float (&b)[kC], float (&win)[kW][kC],
                                           const float (&x)[kC], int silu, uint16_t *out) {
    float pre[kC];
#pragma unroll
    for (int e = 0; e < kC; ++e) win[kW - 1][e] = x[e];
    convolve<kC, kW>(w, b, win, pre);
    if (silu) {
#pragma unroll
        for (int e = 0; e < kC; ++e) pre[e] *= sigmoid(pre[e]);
    }
    store_c<kC>(out, pre);
#pragma unroll
    for (int k = 0; k < kW - 1; ++k)
#pragma unroll
        for (int e = 0; e < kC; ++e) win[k][e] = win[k + 1][e];
}

// The final state of sequence n: its last W - 1 inputs.  All are read before
// the first is written, so that ht may be h0 once nothing else reads that.
template <int kC, int kW>
__device__ __forceinline__ void final_state(const ConvArgs &a, const Seqs &sq, int64_t n, int64_t c) {
    const int64_t begin = sq.begin(n), len = sq.end(n) > begin ? sq.end(n) - begin : 0;
    float v[kW - 1][kC];
#pragma unroll
    for (int j = 0; j < kW - 1; ++j) input_at<kC, kW>(a, n, begin, len - (kW - 1) + j, c, v[j]);
#pragma unroll
    for (int j = 0; j < kW - 1; ++j) store_any_c<kC>(a.ht, (n * (kW - 1) + j) * a.D + c, a.ht_f32, v[j]);
}

// The first state_blocks workgroups along y write final states instead.
template <int kC, int kW>
__global__ __launch_bounds__(kLanes *kWaves) void kda_conv_kernel(ConvArgs a, int state_blocks) {
    const int64_t c = ((int64_t)blockIdx.x * kLanes + (threadIdx.x & 63)) * kC;
    if (c >= a.D) return;
    const Seqs sq = seqs_of(a);
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if ((int)blockIdx.y < state_blocks) {
        for (int64_t n = (int64_t)blockIdx.y * kWaves + wave; n < sq.N; n += (int64_t)state_blocks * kWaves)
            final_state<kC, kW>(a, sq, n, c);
        return;
    }
    const int64_t by = blockIdx.y - state_blocks, blocks = gridDim.y - state_blocks;
    float w[kW][kC], b[kC];
    load_filter<kC, kW>(a, c, w, b);
    const int64_t runs = (a.T + kRun - 1) / kRun;
    for (int64_t u = by * kWaves + wave; u < a.B * runs; u += blocks * kWaves) {
        const Run run = run_of(u, runs, a.T, kRun);
        int64_t n = sq.of(run.t0);
        if (n >= sq.N) return;  // behind the last sequence, and so are later runs
        const uint16_t *xp = a.x + run.b * a.xb + (run.t0 - run.b * a.T) * a.xt + c;
        uint16_t *op = a.out + run.t0 * a.D + c;
        int64_t begin = sq.begin(n), next = sq.end(n);
        float win[kW][kC];     // win[k]: the input k steps after the oldest one that the token needs
        if (run.t0 + kRun <= next && run.t0 + kRun <= run.stop) {
            // the run lies within one sequence: all its loads in flight together
            float x[kRun][kC];
#pragma unroll
            for (int i = 0; i < kRun; ++i) load_c<kC>(xp + i * a.xt, x[i]);
#pragma unroll
            for (int k = 0; k < kW - 1; ++k) input_at<kC, kW>(a, n, begin, run.t0 - begin - (kW - 1) + k, c, win[k]);
#pragma unroll
            for (int i = 0; i < kRun; ++i) conv_token<kC, kW>(w, b, win, x[i], a.silu, op + i * a.D);
            continue;
        }
#pragma unroll
        for (int k = 0; k < kW - 1; ++k) input_at<kC, kW>(a, n, begin, run.t0 - begin - (kW - 1) + k, c, win[k]);
        for (int64_t t = run.t0; t < run.stop; ++t) {
            if (t >= next) {  // the next sequence that has tokens
                do { ++n; } while (n < sq.N && sq.end(n) <= t);
                if (n >= sq.N) break;
                begin = sq.begin(n);
                next = sq.end(n);
#pragma unroll
                for (int k = 0; k < kW - 1; ++k) input_at<kC, kW>(a, n, begin, t - begin - (kW - 1) + k, c, win[k]);
            }
            float x[kC];
            load_c<kC>(xp + (t - run.t0) * a.xt, x);
            conv_token<kC, kW>(w, b, win, x, a.silu, op + (t - run.t0) * a.D);
        }
    }
}

// Final states in a launch of their own, for ht the same as h0.
template <int kC, int kW>
__global__ __launch_bounds__(kLanes *kWaves) void kda_conv_state_kernel(ConvArgs a) {
    const int64_t c = ((int64_t)blockIdx.x * kLanes + (threadIdx.x & 63)) * kC;
    if (c >= a.D) return;
    const Seqs sq = seqs_of(a);
    for (int64_t n = (int64_t)blockIdx.y * kWaves + (threadIdx.x >> 6); n < sq.N; n += (int64_t)gridDim.y * kWaves)
        final_state<kC, kW>(a, sq, n, c);
}

// One token per sequence: output and shifted state in one launch.
template <int kC, int kW>
__global__ __launch_bounds__(64) void kda_conv_decode_kernel(ConvArgs a) {
    const int64_t c = ((int64_t)blockIdx.x * 64 + threadIdx.x) * kC;
    if (c >= a.D) return;
    for (int64_t n = blockIdx.y; n < a.N; n += gridDim.y) {
        float win[kW][kC], w[kW][kC], b[kC], pre[kC];
        load_c<kC>(a.x + n * a.xb + c, win[kW - 1]);
#pragma unroll
        for (int k = 0; k < kW - 1; ++k) input_at<kC, kW>(a, n, 0, k - (kW - 1), c, win[k]);
        load_filter<kC, kW>(a, c, w, b);
        convolve<kC, kW>(w, b, win, pre);
        if (a.silu) {
#pragma unroll
            for (int e = 0; e < kC; ++e) pre[e] *= sigmoid(pre[e]);
        }
        store_c<kC>(a.out + n * a.D + c, pre);
#pragma unroll
        for (int k = 0; k < kW - 1; ++k) store_any_c<kC>(a.ht, (n * (kW - 1) + k) * a.D + c, a.ht_f32, win[k + 1]);
    }
}

// ---- gradient ----------------------------------------------------------------
//
//   dpre_t = d_out_t act'(pre_t),   dx_t = sum_k w_k dpre_{t + (W - 1) - k}
//   (tokens of the same sequence) + d_final_state,   dw_k = sum_t dpre_t x_{t - (W - 1) + k}
//
// A wave walks over its run and W - 1 tokens further, computing pre again; each
// dpre is added to the W pending dx entries it reaches (pend[k] is that of
// token t - (W - 1) + k), and the oldest one is written.  At the end of a
// sequence the pending ones are complete.

// The derivative of the activation, times g.  For silu, with s = sigmoid(p):
// s (1 + p (1 - s)).
__device__ __forceinline__ float act_grad(float p, float g, int silu) {
    if (!silu) return g;
    const float s = sigmoid(p);
    return g * s * (1.0f + p * (1.0f - s));
}

template <int kC, int kW>
struct BwdWalk {
    const ConvArgs &a;
    const Seqs &sq;
    int64_t c, t0, stop;      // the run whose dx this wave writes
    int64_t n, begin, next;
    float pend[kW][kC];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < kW; ++k)
#pragma unroll
            for (int e = 0; e < kC; ++e) pend[k][e] = 0.f;
    }
    // dx of token t, complete but for the final state's share.
    __device__ __forceinline__ void emit(int64_t t, const float *v) {
        if (t < t0 || t >= stop || t < begin) return;
        float o[kC];
#pragma unroll
        for (int e = 0; e < kC; ++e) o[e] = v[e];
        const int64_t j = t - (next - (kW - 1));
        if (a.dht && j >= 0) {
            float d[kC];
            load_any_c<kC>(a.dht, (n * (kW - 1) + j) * a.D + c, a.ht_f32, d);
#pragma unroll
            for (int e = 0; e < kC; ++e) o[e] += d[e];
        }
        store_c<kC>(a.dx + t * a.D + c, o);
    }
    // After the last token, t - 1, of a sequence or of the walk.
    __device__ __forceinline__ void flush(int64_t t) {
#pragma unroll
        for (int k = 0; k < kW - 1; ++k) emit(t - (kW - 1) + k, pend[k]);
    }
};

template <int kC, int kW>
__global__ __launch_bounds__(kLanes *kWaves) void kda_conv_bwd_kernel(ConvArgs a) {
    __shared__ float red[kWaves][kW + 1][kC][kLanes];
    const int lane = threadIdx.x & 63;
    const int64_t c = ((int64_t)blockIdx.x * kLanes + lane) * kC;
    const bool in = c < a.D;
    const Seqs sq = seqs_of(a);
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    float dw[kW + 1][kC];
#pragma unroll
    for (int k = 0; k <= kW; ++k)
#pragma unroll
        for (int e = 0; e < kC; ++e) dw[k][e] = 0.f;
    if (in) {
        float w[kW][kC], b[kC];
        load_filter<kC, kW>(a, c, w, b);
        const int64_t runs = (a.T + kBwdRun - 1) / kBwdRun;
        for (int64_t v = (int64_t)blockIdx.y * kWaves + wave; v < a.B * runs; v += (int64_t)gridDim.y * kWaves) {
            const Run run = run_of(v, runs, a.T, kBwdRun);
            const int64_t t0 = run.t0;
            const uint16_t *xp = a.x + run.b * a.xb + (t0 - run.b * a.T) * a.xt + c;
            const uint16_t *yp = a.dy + run.b * a.db_ + (t0 - run.b * a.T) * a.dt_ + c;
            BwdWalk<kC, kW> s{a, sq, c, t0, run.stop, sq.of(t0), 0, 0, {}};
            if (s.n >= sq.N) break;
            s.clear();
            s.begin = sq.begin(s.n);
            s.next = sq.end(s.n);
            float win[kW][kC];
#pragma unroll
            for (int k = 0; k < kW - 1; ++k) input_at<kC, kW>(a, s.n, s.begin, t0 - s.begin - (kW - 1) + k, c, win[k]);
            int64_t t = t0;
            // unrolled: the next tokens' loads go out while this one is computed
#pragma unroll 4
            for (; t < s.stop + kW - 1; ++t) {
                if (t >= s.next) {
                    s.flush(t);
                    s.clear();
                    if (t >= s.stop) break;
                    do { ++s.n; } while (s.n < sq.N && sq.end(s.n) <= t);
                    if (s.n >= sq.N) break;
                    s.begin = sq.begin(s.n);
                    s.next = sq.end(s.n);
#pragma unroll
                    for (int k = 0; k < kW - 1; ++k) input_at<kC, kW>(a, s.n, s.begin, t - s.begin - (kW - 1) + k, c, win[k]);
                }
                float g[kC], pre[kC];
                load_c<kC>(xp + (t - t0) * a.xt, win[kW - 1]);
                load_c<kC>(yp + (t - t0) * a.dt_, g);
                convolve<kC, kW>(w, b, win, pre);
#pragma unroll
                for (int e = 0; e < kC; ++e) {
                    const float d = act_grad(pre[e], g[e], a.silu);
                    // pend[k] is token t - (W - 1) + k, which tap k of token t reads
#pragma unroll
                    for (int k = 0; k < kW; ++k) s.pend[k][e] += w[k][e] * d;
                    if (t < s.stop) {
#pragma unroll
                        for (int k = 0; k < kW; ++k) dw[k][e] += d * win[k][e];
                        dw[kW][e] += d;
                    }
                }
                s.emit(t - (kW - 1), s.pend[0]);
#pragma unroll
                for (int k = 0; k < kW - 1; ++k)
#pragma unroll
                    for (int e = 0; e < kC; ++e) {
                        win[k][e] = win[k + 1][e];
                        s.pend[k][e] = s.pend[k + 1][e];
                    }
#pragma unroll
                for (int e = 0; e < kC; ++e) s.pend[kW - 1][e] = 0.f;
            }
        }
    }
#pragma unroll
    for (int k = 0; k <= kW; ++k)
#pragma unroll
        for (int e = 0; e < kC; ++e) red[wave][k][e][lane] = dw[k][e];
    __syncthreads();
    if (!in) return;
    for (int k = wave; k <= kW; k += kWaves) {
        float v[kC];
#pragma unroll
        for (int e = 0; e < kC; ++e) {
            v[e] = red[0][k][e][lane];
#pragma unroll
            for (int q = 1; q < kWaves; ++q) v[e] += red[q][k][e][lane];
        }
        store_f32_c<kC>(a.part + ((int64_t)blockIdx.y * (kW + 1) + k) * a.D + c, v);
    }
}

// dweight and dbias: the sum of the partial sums, in a fixed order.  A workgroup
// takes 64 channels of one tap, 16 waves over the parts.
template <int kW>
__global__ __launch_bounds__(1024) void kda_conv_bwd_sum_kernel(ConvArgs a) {
    __shared__ float s[16][64];
    const int lane = threadIdx.x & 63, q = threadIdx.x >> 6, k = blockIdx.y;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float v = 0.f;
    if (c < a.D)
        for (int64_t p = q; p < a.parts; p += 16) v += a.part[(p * (kW + 1) + k) * a.D + c];
    s[q][lane] = v;
    __syncthreads();
    if (q != 0 || c >= a.D) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) v += s[i][lane];
    if (k < kW) a.dw[c * kW + k] = v;
    else if (a.dbias) a.dbias[c] = v;
}

// The initial state's gradient: entry m (input m - (W - 1)) reaches the tokens
// p <= m through tap m - p, and, in a sequence shorter than W - 1, the final
// state's entry m - length.
template <int kC, int kW>
__global__ __launch_bounds__(64) void kda_conv_bwd_state_kernel(ConvArgs a) {
    const int64_t c = ((int64_t)blockIdx.x * 64 + threadIdx.x) * kC;
    if (c >= a.D) return;
    const Seqs sq = seqs_of(a);
    float w[kW][kC], b[kC];
    load_filter<kC, kW>(a, c, w, b);
    for (int64_t n = blockIdx.y; n < sq.N; n += gridDim.y) {
        const int64_t begin = sq.begin(n), len = sq.end(n) > begin ? sq.end(n) - begin : 0;
        float d[kW - 1][kC];
#pragma unroll
        for (int m = 0; m < kW - 1; ++m) {
#pragma unroll
            for (int e = 0; e < kC; ++e) d[m][e] = 0.f;
            if (a.dht && m >= len) load_any_c<kC>(a.dht, (n * (kW - 1) + m - len) * a.D + c, a.ht_f32, d[m]);
        }
#pragma unroll
        for (int p = 0; p < kW - 1; ++p) {
            if (p >= len) break;
            float win[kW][kC], g[kC], pre[kC];
#pragma unroll
            for (int k = 0; k < kW; ++k) input_at<kC, kW>(a, n, begin, p - (kW - 1) + k, c, win[k]);
            load_c<kC>(a.dy + row_of(begin + p, a.T, a.db_, a.dt_) + c, g);
            convolve<kC, kW>(w, b, win, pre);
#pragma unroll
            for (int e = 0; e < kC; ++e) {
                const float dp = act_grad(pre[e], g[e], a.silu);
#pragma unroll
                for (int m = p; m < kW - 1; ++m) d[m][e] += w[m - p][e] * dp;
            }
        }
#pragma unroll
        for (int m = 0; m < kW - 1; ++m) store_f32_c<kC>(a.dh0 + (n * (kW - 1) + m) * a.D + c, d[m]);
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Wide accesses to every tensor of the call.  Stricter than they need: a lane's 4
// channels are 8 bytes of bf16 and 16 of fp32, so multiples of 4 channels at 8-byte
// addresses (fp32: 16) would do (8192 tokens of 4352 channels 31 us, of 4356 45).
bool vector_channels(const ConvArgs &a) {
    return a.D % 8 == 0 && a.xb % 8 == 0 && a.xt % 8 == 0 && a.db_ % 8 == 0 && a.dt_ % 8 == 0 && aligned16(a.x) &&
           aligned16(a.out) && aligned16(a.h0) && aligned16(a.ht) && aligned16(a.dy) && aligned16(a.dht) &&
           aligned16(a.dx) && aligned16(a.dh0) && aligned16(a.w) && aligned16(a.bias);
}

unsigned blocks_x(int64_t D, int kC, int lanes) { return (unsigned)((D + (int64_t)kC * lanes - 1) / ((int64_t)kC * lanes)); }
unsigned blocks_y(int64_t n, int64_t per) {
    const int64_t b = (n + per - 1) / per;
    return (unsigned)(b < 1 ? 1 : b < kMaxGridY ? b : kMaxGridY);
}

// Sequences per workgroup of final states: with few, one wave each.
constexpr int kMaxStateBlocks = 1024;

template <int kC, int kW>
hipError_t launch_conv(const ConvArgs &a, hipStream_t s) {
    const unsigned x = blocks_x(a.D, kC, kLanes);
    // where the final state replaces the initial one, the tokens read that first
    const bool apart = a.ht && (a.ht == a.h0 || a.B * a.T == 0);
    unsigned states = a.ht ? blocks_y(a.N, kWaves) : 0;
    if (states > kMaxStateBlocks) states = kMaxStateBlocks;
    if (a.B * a.T > 0) {
        const unsigned y = blocks_y(a.B * ((a.T + kRun - 1) / kRun), kWaves);
        const unsigned first = apart ? 0 : states;
        hipLaunchKernelGGL((kda_conv_kernel<kC, kW>), dim3(x, first + (y < kMaxGridY - first ? y : (unsigned)kMaxGridY - first)),
                           dim3(kLanes * kWaves), 0, s, a, (int)first);
    }
    if (apart) hipLaunchKernelGGL((kda_conv_state_kernel<kC, kW>), dim3(x, states), dim3(kLanes * kWaves), 0, s, a);
    return hipGetLastError();
}

template <int kC, int kW>
hipError_t launch_conv_bwd(const ConvArgs &a, hipStream_t s) {
    ConvArgs b = a;
    if (a.B * a.T > 0)
        hipLaunchKernelGGL((kda_conv_bwd_kernel<kC, kW>), dim3(blocks_x(a.D, kC, kLanes), (unsigned)a.parts),
                           dim3(kLanes * kWaves), 0, s, a);
    else b.parts = 0;
    hipLaunchKernelGGL((kda_conv_bwd_sum_kernel<kW>), dim3(blocks_x(a.D, 1, 64), kW + 1), dim3(1024), 0, s, b);
    if (a.dh0)
        hipLaunchKernelGGL((kda_conv_bwd_state_kernel<kC, kW>), dim3(blocks_x(a.D, kC, 64), blocks_y(a.N, 1)), dim3(64), 0, s, a);
    return hipGetLastError();
}

template <int kC, int kW>
hipError_t launch_decode(const ConvArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((kda_conv_decode_kernel<kC, kW>), dim3(blocks_x(a.D, kC, 64), blocks_y(a.N, 1)), dim3(64), 0, s, a);
    return hipGetLastError();
}

}  // namespace

// Channels per lane where 16- and 8-byte accesses are possible.  4 rather than 8:
// half the registers (filter, window, pending sums), twice the waves: the same time
// for prompts, 5% less packed (32768 x 4352), 66 against 79 us for the gradient of
// 8192 x 4352 when they were compared.
constexpr int kVec = 4;

#define KDA_CONV_DISPATCH(fn)                                                          \
    if (vector_channels(a)) return W == 2 ? fn<kVec, 2>(a, s) : W == 3 ? fn<kVec, 3>(a, s) : fn<kVec, 4>(a, s); \
    return W == 2 ? fn<1, 2>(a, s) : W == 3 ? fn<1, 3>(a, s) : fn<1, 4>(a, s)

hipError_t kda_launch_conv(const ConvArgs &a, int W, hipStream_t s) { KDA_CONV_DISPATCH(launch_conv); }

hipError_t kda_launch_conv_decode(const ConvArgs &a, int W, hipStream_t s) { KDA_CONV_DISPATCH(launch_decode); }

// Workgroups along the tokens of the gradient, each of which writes a partial
// sum of dweight and dbias.
int64_t kda_conv_parts(int64_t B, int64_t T, int64_t D) {
    (void)D;
    const int64_t n = (B * ((T + kBwdRun - 1) / kBwdRun) + kWaves - 1) / kWaves;
    return n < 1 ? 1 : n < 256 ? n : 256;
}

hipError_t kda_launch_conv_bwd(const ConvArgs &a, int W, hipStream_t s) { KDA_CONV_DISPATCH(launch_conv_bwd); }
