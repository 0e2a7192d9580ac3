// kda_ssm_decode.hip -- one step of the selective state-space scan per
// sequence (gfx950).
//
//   S' = exp(-exp(A_log) dt) S + dt x B^T,   y = S' C + D x,   dt = softplus(. + dt_bias)
//
// The state is read once, updated in registers and written once, in fp32
// arithmetic: the step is bound by the state's memory traffic (64 KiB in and
// out per head of 64 x 128 fp32).  64 sequences of 64 heads, 268 MB: 49 us from states
// that are not resident and 52 in place (5.5 and 5.1 TB/s), 40 from ones that the
// caches kept from the step before; 256 sequences 180 us (6.0 TB/s, a copy's rate).
//
// A workgroup of 256 threads takes kRows rows (channels) of one head's state; a
// thread holds 4 neighbouring columns of every 256 / (N / 4)-th row, so that a
// row is one contiguous access of N / 4 lanes, whose shares of S' C are added by
// lane exchanges.  32 rows, so that a few sequences fill the GPU (one sequence of
// 64 heads of 64 x 128 fp32: 4.3 us against 5.6 with 64 rows).
#include "kda_layer_args.h"

using namespace kda;

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 32;

// The new state is stored with the non-temporal hint: it displaces less of what
// the caches still hold of the state being read (64 sequences of 64 heads, 128 MiB
// into another tensor: 45 us against 54; in place 41 against 44).  States that do
// not fit the 256 MB Infinity Cache at all are read past it as well (256
// sequences, 512 MiB, in place: 181 us against 199); at 256 MiB and below that
// costs more than it gives (128 sequences: 93 us against 79).
constexpr int64_t kStreamBytes = 384ll << 20;

typedef uint32_t u2v __attribute__((ext_vector_type(2)));

template <bool kStream, typename T>
__device__ __forceinline__ T state_load(const T *p) {
    if constexpr (kStream) return __builtin_nontemporal_load(p);
    else return *p;
}
template <bool kStream>
__device__ __forceinline__ f4 load_state4(const void *p, int64_t i, int f32) {
    if (f32) return state_load<kStream>(reinterpret_cast<const f4 *>(reinterpret_cast<const float *>(p) + i));
    const u2v v = state_load<kStream>(reinterpret_cast<const u2v *>(reinterpret_cast<const uint16_t *>(p) + i));
    return f4{__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xffff0000u), __uint_as_float(v[1] << 16),
              __uint_as_float(v[1] & 0xffff0000u)};
}
__device__ __forceinline__ void store_state4(void *p, int64_t i, int f32, f4 v) {
    if (f32) __builtin_nontemporal_store(v, reinterpret_cast<f4 *>(reinterpret_cast<float *>(p) + i));
    else
        __builtin_nontemporal_store(u2v{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])},
                                    reinterpret_cast<u2v *>(reinterpret_cast<uint16_t *>(p) + i));
}

template <int kN, bool kStream>
__global__ __launch_bounds__(kThreads) void kda_ssm_decode_kernel(SsmArgs a, int64_t base_block) {
    constexpr int kCols = kN / 4;                // threads per row
    constexpr int kStep = kThreads / kCols;      // rows per pass
    constexpr int kPass = kRows / kStep;
    static_assert(kRows % kStep == 0, "whole passes");
    const int share = (int)(a.P / kRows);
    const int64_t block = base_block + blockIdx.x;
    const int64_t unit = block / share;          // (sequence, head)
    const int p0 = (int)(block - unit * share) * kRows;
    const int64_t n = unit / a.H, h = unit - n * a.H;
    const int64_t g = h / (a.H / a.G);
    const int q = threadIdx.x % kCols, r = threadIdx.x / kCols;
    const int64_t base = (unit * a.P + p0 + r) * kN + 4 * q;
    f4 S[kPass];
#pragma unroll
    for (int i = 0; i < kPass; ++i)
        S[i] = a.h0 ? load_state4<kStream>(a.h0, base + (int64_t)i * kStep * kN, a.h0_f32) : f4{0.f, 0.f, 0.f, 0.f};
    const f4 Bv = load_state4<false>(a.Bm, n * a.bb + g * kN + 4 * q, 0);
    const f4 Cv = load_state4<false>(a.Cm, n * a.cb + g * kN + 4 * q, 0);
    const float raw = bf16_bits_to_f32(a.dt[n * a.dtb + h]) + (a.dt_bias ? a.dt_bias[h] : 0.f);
    const float dt = softplus(raw);
    const float decay = exact_exp(-decay_rate(a.A_log[h]) * dt);
    const float Dh = a.D ? a.D[h] : 0.f;
    const uint16_t *x = a.x + n * a.xb + h * a.P + p0;
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
        const float xv = bf16_bits_to_f32(x[i * kStep + r]);
        const float dx = dt * xv;
        float y = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            S[i][e] = decay * S[i][e] + dx * Bv[e];
            y += S[i][e] * Cv[e];
        }
        store_state4(a.ht, base + (int64_t)i * kStep * kN, a.ht_f32, S[i]);
#pragma unroll
        for (int m = kCols / 2; m >= 1; m >>= 1) y += __shfl_xor(y, m);
        if (q == 0) a.out[unit * a.P + p0 + i * kStep + r] = f32_to_bf16_bits(y + Dh * xv);
    }
}

template <int kN, bool kStream>
hipError_t launch(const SsmArgs &a, hipStream_t s) {
    return launch_groups(a.num_seqs * a.H * (a.P / kRows), a.launch_cap, [&](int64_t base, dim3 grid) {
        hipLaunchKernelGGL((kda_ssm_decode_kernel<kN, kStream>), grid, dim3(kThreads), 0, s, a, base);
    });
}

}  // namespace

hipError_t kda_launch_ssm_decode(const SsmArgs &a, hipStream_t s) {
    const bool stream = a.num_seqs * a.H * a.P * a.N * (a.h0_f32 ? 4 : 2) >= kStreamBytes;
    if (a.N == 128) return stream ? launch<128, true>(a, s) : launch<128, false>(a, s);
    return stream ? launch<64, true>(a, s) : launch<64, false>(a, s);
}
