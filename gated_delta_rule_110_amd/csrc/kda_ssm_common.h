// kda_ssm_common.h -- what the scan's kernels share (kda_ssm.hip, kda_ssm_bwd.hip):
// chunks, LDS layout, the transposing read, operand splits, step sizes.
#pragma once
#include "kda_layer_args.h"

namespace kda {

constexpr int kL = 64;        // tokens per chunk
constexpr int kPB = 64;       // channels per workgroup
constexpr float kLog2e = 1.4426950408889634f;

typedef short s4 __attribute__((ext_vector_type(4)));

// LDS rows are padded: 64 bytes behind the N values of B and C, 32 behind the
// 64 channels of x, so that the 16 rows (and 4-row groups of the transposing
// read) of one access spread over the banks.
template <int kN> constexpr int kPitch = kN + 32;
constexpr int kXPitch = kPB + 16;

// The transposing read: within 16 lanes, lane l gives the address of 4 values
// and receives, as entry e, value l % 4 of those that lane 4 e + l / 4 addressed.
// Two of them give a lane the 8 tokens 4 g + e and 16 + 4 g + e (e < 4) of one
// column, the token order in which accumulators of 16 x 16 products hold them.
__device__ __forceinline__ s4 read_tr(const uint16_t *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s4 *)(__attribute__((address_space(3))) void *)const_cast<uint16_t *>(p));
}
__device__ __forceinline__ s8 join(s4 a, s4 b) { return s8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}; }

__device__ __forceinline__ s8 lds8(const uint16_t *p) { return *reinterpret_cast<const s8 *>(p); }

__device__ __forceinline__ int64_t clamp_to(int64_t v, int64_t hi) { return v < 0 ? 0 : v > hi ? hi : v; }

// Rows of kN (or 64) bf16 values to registers and on to LDS: 16 bytes a thread.
template <int kCols, int kThreads>
struct Rows {
    static constexpr int kPer = kThreads / (kCols / 8);  // rows per pass
    static constexpr int kPass = kL / kPer;
    uint4 v[kPass];
    __device__ __forceinline__ void load(const uint16_t *base, int64_t stride, int rows) {
        const int c = threadIdx.x % (kCols / 8), r = threadIdx.x / (kCols / 8);
#pragma unroll
        for (int i = 0; i < kPass; ++i) {
            const int t = i * kPer + r;
            v[i] = make_uint4(0, 0, 0, 0);  // rows behind the sequence count as zero
            if (t < rows) v[i] = *reinterpret_cast<const uint4 *>(base + t * stride + 8 * c);
        }
    }
    __device__ __forceinline__ void store(uint16_t *lds, int pitch) const {
        const int c = threadIdx.x % (kCols / 8), r = threadIdx.x / (kCols / 8);
#pragma unroll
        for (int i = 0; i < kPass; ++i) *reinterpret_cast<uint4 *>(lds + (i * kPer + r) * pitch + 8 * c) = v[i];
    }
};

// Two- and three-part bf16 splits of fp32 values, 8 at a time.
__device__ __forceinline__ void split2(const float *x, s8 &hi, s8 &lo) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        short h, l;
        split_bf16(x[j], h, l);
        hi[j] = h;
        lo[j] = l;
    }
}
__device__ __forceinline__ float bf16_rest(float x, short &hi) {
    hi = (short)f32_to_bf16_bits(x);
    return x - bf16_bits_to_f32((uint16_t)hi);
}
__device__ __forceinline__ void split3(const float *x, s8 &a, s8 &b, s8 &c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        short h, m;
        const float r = bf16_rest(bf16_rest(x[j], h), m);
        a[j] = h;
        b[j] = m;
        c[j] = (short)f32_to_bf16_bits(r);
    }
}

// The chunk's step sizes and running log-decays, by wave 0, lane = token.  The
// sums run in 64 bits and are kept as a rounded value and its rest: decays
// between neighbours far into a chunk are differences of large sums (hundreds,
// where the steps are large), and would lose the low bits of fp32 otherwise.
__device__ __forceinline__ void step_sizes(float raw, bool live, float bias, float nA2, float *g, float *gr, float *dts) {
    const float dt = live ? softplus(raw + bias) : 0.f;
    double s = (double)nA2 * (double)dt;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double o = __shfl_up(s, d);
        if (lane >= d) s += o;
    }
    const float hi = (float)s;
    g[lane] = hi;
    gr[lane] = (float)(s - (double)hi);
    dts[lane] = dt;
}

}  // namespace kda
