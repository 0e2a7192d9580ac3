// kda_ssm_common.h -- what the scan's kernels share (kda_ssm.hip, kda_ssm_bwd.hip):
// chunks, LDS layout, the transposing read, operand splits, step sizes.
#pragma once
#include "kda_layer_args.h"

namespace kda {

constexpr int kL = 64;        // tokens per chunk
constexpr int kPB = 64;       // channels per workgroup
constexpr float kLog2e = 1.4426950408889634f;

typedef short s4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));

// LDS rows are padded by 32 bytes, so that the 16 rows (and the 8-row groups of
// the transposing read) of one access spread over the banks.
template <int kN> constexpr int kPitch = kN + 16;
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

// 64 token rows of kCols bf16 values to registers and on to LDS, 16 bytes a
// thread and pass.  Rows behind the sequence count as zero: they are given an
// offset outside the buffer, for which the hardware loads zeros.  No branch
// around the loads: where paths with different loads meet, the compiler has to
// wait for all that may be in flight, stores included (the outputs' pass over
// 8192 x 64 heads lost 1500 of 8600 cycles a chunk to that).
template <int kCols, int kThreads>
struct Rows {
    static constexpr int kPer = kThreads / (kCols / 8);  // rows per pass
    static constexpr int kPass = kL / kPer;
    static constexpr uint32_t kSize = 0x7ffffff0u;       // above 64 rows of 2^24 entries
    u4v v[kPass];
    uint32_t off;                                        // bytes from a pass's first row
    uint32_t step;                                       // bytes between the passes
    int r, lds;
    // The host refuses token strides of 2^24 entries and more.
    __device__ __forceinline__ void init(int64_t stride, int pitch) {
        const int thread = threadIdx.x % kThreads;       // larger workgroups: a set of rows per kThreads of them
        const int c = thread % (kCols / 8);
        r = thread / (kCols / 8);
        off = ((uint32_t)r * (uint32_t)stride + 8 * c) * 2;
        step = kPer * (uint32_t)stride * 2;
        lds = r * pitch + 8 * c;
    }
    __device__ __forceinline__ void load(const uint16_t *base, int rows) {
        // a raw buffer of bytes: no stride, no swizzle
        const auto buffer = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(base), 0, kSize, 0x00020000);
#pragma unroll
        for (int i = 0; i < kPass; ++i)
            v[i] = __builtin_amdgcn_raw_buffer_load_b128(buffer, i * kPer + r < rows ? off : kSize, i * step, 0);
    }
    __device__ __forceinline__ void store(uint16_t *to, int pitch) const {
#pragma unroll
        for (int i = 0; i < kPass; ++i) *reinterpret_cast<u4v *>(to + i * kPer * pitch + lds) = v[i];
    }
};

// Splits of fp32 values into three bf16 parts (24 bits, fp32's own), each rounded to
// nearest and the next taken from what it left, two values at a time.
constexpr int kParts = 3;
typedef float f2v __attribute__((ext_vector_type(2)));
typedef __bf16 b2v __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t round_pair(float &a, float &b) {
    const uint32_t h = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2v{a, b}, b2v));
    a -= __uint_as_float(h << 16);
    b -= __uint_as_float(h & 0xffff0000u);
    return h;
}
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2v{a, b}, b2v));
}
__device__ __forceinline__ void split3(const float *x, s8 &p, s8 &q, s8 &r) {
    u4v h, m, l;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a = x[2 * j], b = x[2 * j + 1];
        h[j] = round_pair(a, b);
        m[j] = round_pair(a, b);
        l[j] = pack_pair(a, b);
    }
    p = __builtin_bit_cast(s8, h);
    q = __builtin_bit_cast(s8, m);
    r = __builtin_bit_cast(s8, l);
}
// Four values in their parts, `apart` entries from each other.
__device__ __forceinline__ void keep_parts(float (&v)[4], uint16_t *to, int apart) {
#pragma unroll
    for (int part = 0; part < kParts - 1; ++part) {
        const uint32_t h0 = round_pair(v[0], v[1]), h1 = round_pair(v[2], v[3]);
        *reinterpret_cast<uint2 *>(to + part * apart) = make_uint2(h0, h1);
    }
    *reinterpret_cast<uint2 *>(to + (kParts - 1) * apart) = make_uint2(pack_pair(v[0], v[1]), pack_pair(v[2], v[3]));
}

// Inclusive running sum over the 64 lanes, in 64 bits: within rows of 16 lanes,
// then the rows before (lane moves only, no LDS).
template <int kCtrl, int kRows>
__device__ __forceinline__ double lane_move(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, kCtrl, kRows, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), kCtrl, kRows, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_scan(double v) {
    v += lane_move<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8: lanes without a source add 0
    v += lane_move<0x112, 0xf>(v);
    v += lane_move<0x114, 0xf>(v);
    v += lane_move<0x118, 0xf>(v);
    v += lane_move<0x142, 0xa>(v);  // the last lane of rows 0 and 2 to rows 1 and 3
    v += lane_move<0x143, 0xc>(v);  // lane 31 to rows 2 and 3
    return v;
}

// The chunk's step sizes and running log-decays (base 2), by one wave, lane =
// token.  The sums run in 64 bits and are kept as a rounded value and its rest:
// decays between neighbours far into a chunk are differences of large sums
// (hundreds, where the steps are large), and would lose the low bits of fp32.
struct Steps {
    float g[kL], gr[kL];          // log2 of the decay from the chunk's start: value and rest
    float dt[kL];
    float from[kL];               // the decay itself, from the chunk's start
    float w[kL];                  // the decay to the chunk's end, times dt
};
__device__ __forceinline__ void step_sizes(float raw, bool live, float bias, float nA2, Steps &o) {
    const float dt = live ? softplus(raw + bias) : 0.f;
    const double s = wave_scan((double)nA2 * (double)dt);
    const int lane = threadIdx.x & 63;
    const float hi = (float)s;
    const uint64_t u = __builtin_bit_cast(uint64_t, s);
    const uint64_t e = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), 63) << 32 |
                       (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63);
    o.g[lane] = hi;
    o.gr[lane] = (float)(s - (double)hi);
    o.dt[lane] = dt;
    o.from[lane] = __builtin_amdgcn_exp2f(hi);
    o.w[lane] = __builtin_amdgcn_exp2f((float)(__builtin_bit_cast(double, e) - s)) * dt;
}

}  // namespace kda
