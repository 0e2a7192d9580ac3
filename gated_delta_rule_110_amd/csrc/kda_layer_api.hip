// kda_layer_api.hip -- the C ABI of the layer operators (include/kda_layer.h):
// validation, workspaces, launches.
#include <math.h>
#include <stdlib.h>
#include <new>
#include <vector>
#include "kda_layer.h"
#include "kda_layer_args.h"

using namespace kda;

namespace {

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool dtype_ok(int32_t d) { return d == KDA_BF16 || d == KDA_FP32; }
size_t width(int32_t d) { return d == KDA_FP32 ? 4 : 2; }

// Sizes beyond these are refused, so that no product of a call's sizes passes
// 63 bits (rows and columns) or a grid's 2^31 - 1 workgroups.
constexpr int64_t kMaxTokens = int64_t(1) << 40;
constexpr int64_t kMaxColumns = int64_t(1) << 22;
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxTokenStride = int64_t(1) << 24;
constexpr int64_t kMaxSeqs = 0x7fffffff;
constexpr int64_t kMaxScanTokens = (int64_t(1) << 31) - 128;  // pieces and chunks are counted in 32 bits

bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }

// The memory a call touches: every written tensor has to lie apart from all
// others, but for a read tensor that it may be one and the same as.
class Memory {
public:
    // `bytes` from the first element to behind the last (0: nothing is touched).
    void read(const void *p, size_t bytes) { add(p, bytes, false, nullptr); }
    void write(const void *p, size_t bytes, const void *may_be = nullptr) { add(p, bytes, true, may_be); }
    bool clash() const {
        for (int i = 0; i < n_; ++i)
            for (int j = 0; j < n_; ++j) {
                const Span &w = s_[i], &o = s_[j];
                if (i == j || !w.written || w.a >= o.b || o.a >= w.b) continue;
                if (!o.written && w.may_be == o.a && w.a == o.a && w.b == o.b) continue;
                return true;
            }
        return false;
    }

private:
    struct Span {
        uintptr_t a, b, may_be;
        bool written;
    };
    void add(const void *p, size_t bytes, bool written, const void *may_be) {
        if (!p || !bytes) return;
        const uintptr_t a = reinterpret_cast<uintptr_t>(p);
        s_[n_++] = Span{a, a + bytes, reinterpret_cast<uintptr_t>(may_be), written};
    }
    Span s_[24];  // more than any call has tensors
    int n_ = 0;
};

// Bytes from the first element of [n0, n1, inner] with strides s0, s1 to behind its last.
size_t extent(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t inner, size_t w) {
    if (n0 <= 0 || n1 <= 0 || inner <= 0) return 0;
    return (size_t)((n0 - 1) * s0 + (n1 - 1) * s1 + inner) * w;
}

// The workspace of a call: the caller's, or one taken on the stream and given
// back behind the call's kernels.
class Workspace {
public:
    Workspace(void *given, size_t bytes, size_t need, hipStream_t s) : p_(given), s_(s) {
        if (need == 0) return;
        if (given) {
            status_ = !aligned(given, 256) ? KDA_ERR_ALIGN : bytes < need ? KDA_ERR_WORKSPACE : KDA_OK;
        } else {
            owned_ = hipMallocAsync(&p_, need, s) == hipSuccess;
            if (!owned_) status_ = KDA_ERR_HIP;
        }
    }
    ~Workspace() {
        if (owned_) (void)hipFreeAsync(p_, s_);
    }
    Workspace(const Workspace &) = delete;
    Workspace &operator=(const Workspace &) = delete;
    kda_status_t status() const { return status_; }
    char *at(size_t off) const { return static_cast<char *>(p_) + off; }

private:
    void *p_;
    hipStream_t s_;
    bool owned_ = false;
    kda_status_t status_ = KDA_OK;
};

kda_status_t of_hip(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

// KDA_VALIDATE=1: the contents of cu_seqlens, read back to the host.
kda_status_t validate_cu(const int64_t *cu, int64_t N, int64_t T, hipStream_t stream) {
    const char *e = getenv("KDA_VALIDATE");
    if (!cu || !(e && e[0] == '1' && e[1] == 0)) return KDA_OK;
    int64_t *h = new (std::nothrow) int64_t[(size_t)N + 1];
    if (!h) return KDA_ERR_HIP;
    kda_status_t st = KDA_OK;
    if (hipMemcpyAsync(h, cu, sizeof(int64_t) * (size_t)(N + 1), hipMemcpyDeviceToHost, stream) != hipSuccess ||
        hipStreamSynchronize(stream) != hipSuccess) {
        st = KDA_ERR_HIP;
    } else {
        if (h[0] != 0 || h[N] > T) st = KDA_ERR_SHAPE;
        for (int64_t n = 0; n < N && st == KDA_OK; ++n)
            if (h[n + 1] < h[n]) st = KDA_ERR_SHAPE;
    }
    delete[] h;
    return st;
}

// ---- RMS normalisation ----

kda_status_t check_norm(const kda_rmsnorm_desc_t *d) {
    if (d->rows < 0 || d->D < 1 || d->rows > kMaxTokens || d->D > kMaxColumns) return KDA_ERR_SHAPE;
    // a smaller eps, which a row of zeros leaves by itself, is zero to the hardware's reciprocal root
    if (!(d->eps >= 0x1p-126f) || !isfinite(d->eps)) return KDA_ERR_PARAM;
    if (!stride_ok(d->x_stride)) return KDA_ERR_SHAPE;
    if (!dtype_ok(d->weight_dtype)) return KDA_ERR_DTYPE;
    return KDA_OK;
}

kda_status_t norm_impl(const void *x, const void *residual, const void *weight, void *residual_out, void *out,
                       float *scales, int quant, const kda_rmsnorm_desc_t *d, hipStream_t stream) {
    if (!d || !weight) return KDA_ERR_NULL;
    const kda_status_t st = check_norm(d);
    if (st != KDA_OK) return st;
    if (d->rows > 0 && (!x || !out || (quant && !scales))) return KDA_ERR_NULL;
    if (residual_out && !residual) return KDA_ERR_NULL;
    if (residual && !dtype_ok(d->residual_dtype)) return KDA_ERR_DTYPE;
    if (residual && !stride_ok(d->residual_stride)) return KDA_ERR_SHAPE;
    if (!aligned(x, 2) || (!quant && !aligned(out, 2)) || !aligned(scales, 4) || !aligned(weight, width(d->weight_dtype)) ||
        (residual && (!aligned(residual, width(d->residual_dtype)) || !aligned(residual_out, width(d->residual_dtype)))))
        return KDA_ERR_ALIGN;
    const size_t n = (size_t)d->rows * (size_t)d->D, rw = width(d->residual_dtype);
    const int64_t groups = d->group ? (d->D + d->group - 1) / d->group : 1;
    Memory m;
    m.read(x, extent(1, 0, d->rows, d->x_stride, d->D, 2));
    if (residual) m.read(residual, extent(1, 0, d->rows, d->residual_stride, d->D, rw));
    m.read(weight, (size_t)d->D * width(d->weight_dtype));
    m.write(out, n * (quant ? 1 : 2), quant ? nullptr : x);
    m.write(residual_out, n * rw, residual);
    m.write(scales, (size_t)d->rows * (size_t)groups * 4);
    if (m.clash()) return KDA_ERR_OVERLAP;
    NormArgs a{};
    a.x = static_cast<const uint16_t *>(x);
    a.res = residual; a.w = weight; a.res_out = residual_out; a.out = out; a.scales = scales;
    a.rows = d->rows; a.D = d->D; a.xs = d->x_stride; a.rs = d->residual_stride;
    a.groups = groups;
    a.eps = d->eps;
    a.res_f32 = d->residual_dtype == KDA_FP32;
    a.w_f32 = d->weight_dtype == KDA_FP32;
    a.quant = !quant ? 0 : d->group ? 2 : 1;
    return of_hip(kda_launch_rmsnorm(a, stream));
}

// ---- short convolution ----

struct ConvShape {
    ConvArgs a;
    size_t need;
};

kda_status_t check_conv(const kda_conv_desc_t *d, bool packed) {
    if (d->B < 1 || d->T < 0 || d->D < 1 || d->num_seqs < 1) return KDA_ERR_SHAPE;
    if (d->B > kMaxSeqs || d->num_seqs > kMaxSeqs || d->T > kMaxTokens / d->B || d->D > kMaxColumns) return KDA_ERR_SHAPE;
    if (packed ? d->B != 1 : d->num_seqs != d->B) return KDA_ERR_SHAPE;
    if (d->W < 2 || d->W > 4) return KDA_ERR_UNSUPPORTED;
    if (d->silu != 0 && d->silu != 1) return KDA_ERR_PARAM;
    if (!stride_ok(d->x_stride_b) || !stride_ok(d->x_stride_t)) return KDA_ERR_SHAPE;
    if (!dtype_ok(d->weight_dtype)) return KDA_ERR_DTYPE;
    return KDA_OK;
}

// What the three calls have in common.
kda_status_t conv_args(const void *x, const void *weight, const void *bias, const void *h0, const void *ht,
                       const int64_t *cu, const kda_conv_desc_t *d, ConvArgs &a) {
    if (!d || !weight) return KDA_ERR_NULL;
    const kda_status_t st = check_conv(d, cu != nullptr);
    if (st != KDA_OK) return st;
    if (d->T > 0 && !x) return KDA_ERR_NULL;
    if (h0 && !dtype_ok(d->initial_state_dtype)) return KDA_ERR_DTYPE;
    if (ht && !dtype_ok(d->final_state_dtype)) return KDA_ERR_DTYPE;
    if (!aligned(x, 2) || !aligned(weight, width(d->weight_dtype)) || !aligned(bias, width(d->weight_dtype)) ||
        (h0 && !aligned(h0, width(d->initial_state_dtype))) || (ht && !aligned(ht, width(d->final_state_dtype))) ||
        !aligned(cu, 8))
        return KDA_ERR_ALIGN;
    a = ConvArgs{};
    a.x = static_cast<const uint16_t *>(x);
    a.w = weight; a.bias = bias; a.h0 = h0; a.cu = cu;
    a.B = d->B; a.T = d->T; a.D = d->D; a.N = d->num_seqs;
    a.xb = d->x_stride_b; a.xt = d->x_stride_t;
    a.silu = d->silu;
    a.w_f32 = d->weight_dtype == KDA_FP32;
    a.h0_f32 = d->initial_state_dtype == KDA_FP32;
    a.ht_f32 = d->final_state_dtype == KDA_FP32;
    return KDA_OK;
}

// What the three calls read; the states' bytes are the same for both.
size_t conv_state_bytes(const kda_conv_desc_t *d, int32_t dtype) {
    return (size_t)d->num_seqs * (size_t)(d->W - 1) * (size_t)d->D * width(dtype);
}
void conv_reads(Memory &m, const void *x, const void *weight, const void *bias, const void *h0, const int64_t *cu,
                const kda_conv_desc_t *d) {
    m.read(x, extent(d->B, d->x_stride_b, d->T, d->x_stride_t, d->D, 2));
    m.read(weight, (size_t)(d->D * d->W) * width(d->weight_dtype));
    m.read(bias, (size_t)d->D * width(d->weight_dtype));
    m.read(h0, conv_state_bytes(d, d->initial_state_dtype));
    m.read(cu, (size_t)(d->num_seqs + 1) * 8);
}
size_t conv_token_bytes(const kda_conv_desc_t *d) { return (size_t)(d->B * d->T) * (size_t)d->D * 2; }

// ---- state-space scan ----

kda_status_t check_ssm(const kda_ssm_desc_t *d, bool packed) {
    if (d->B < 1 || d->T < 0 || d->H < 1 || d->G < 1 || d->num_seqs < 1) return KDA_ERR_SHAPE;
    if (d->H > 65535 || d->H % d->G != 0) return KDA_ERR_SHAPE;
    if (d->B > kMaxSeqs || d->num_seqs > kMaxSeqs || d->T > kMaxScanTokens / d->B) return KDA_ERR_SHAPE;
    if (packed ? d->B != 1 : d->num_seqs != d->B) return KDA_ERR_SHAPE;
    if ((d->P != 64 && d->P != 128) || (d->N != 64 && d->N != 128)) return KDA_ERR_UNSUPPORTED;
    const int64_t strides[] = {d->x_stride_b, d->x_stride_t, d->dt_stride_b, d->dt_stride_t,
                               d->b_stride_b, d->b_stride_t, d->c_stride_b, d->c_stride_t};
    for (int64_t s : strides)
        if (!stride_ok(s)) return KDA_ERR_SHAPE;
    // the offsets of a chunk's tokens are kept in 32 bits
    for (int64_t s : {d->x_stride_t, d->dt_stride_t, d->b_stride_t, d->c_stride_t})
        if (s >= kMaxTokenStride) return KDA_ERR_SHAPE;
    // x, B and C are read 16 bytes at a time
    for (int64_t s : {d->x_stride_b, d->x_stride_t, d->b_stride_b, d->b_stride_t, d->c_stride_b, d->c_stride_t})
        if (s % 8 != 0) return KDA_ERR_ALIGN;
    if (d->piece_chunks < 0 || d->launch_piece < 0) return KDA_ERR_PARAM;
    return KDA_OK;
}

kda_status_t ssm_args(const void *x, const void *dt, const void *Bm, const void *Cm, const float *A_log,
                      const float *dt_bias, const float *D, const void *h0, const void *ht, const int64_t *cu,
                      const kda_ssm_desc_t *d, SsmArgs &a) {
    if (!d || !A_log) return KDA_ERR_NULL;
    const kda_status_t st = check_ssm(d, cu != nullptr);
    if (st != KDA_OK) return st;
    if (d->T > 0 && (!x || !dt || !Bm || !Cm)) return KDA_ERR_NULL;
    if (h0 && !dtype_ok(d->initial_state_dtype)) return KDA_ERR_DTYPE;
    if (ht && !dtype_ok(d->final_state_dtype)) return KDA_ERR_DTYPE;
    if (!aligned(x, 16) || !aligned(Bm, 16) || !aligned(Cm, 16) || !aligned(h0, 16) || !aligned(ht, 16) || !aligned(dt, 2) ||
        !aligned(A_log, 4) || !aligned(dt_bias, 4) || !aligned(D, 4) || !aligned(cu, 8))
        return KDA_ERR_ALIGN;
    a = SsmArgs{};
    a.x = static_cast<const uint16_t *>(x);
    a.dt = static_cast<const uint16_t *>(dt);
    a.Bm = static_cast<const uint16_t *>(Bm);
    a.Cm = static_cast<const uint16_t *>(Cm);
    a.A_log = A_log; a.dt_bias = dt_bias; a.D = D; a.h0 = h0; a.cu = cu;
    a.B = d->B; a.T = d->T; a.H = d->H; a.P = d->P; a.G = d->G; a.N = d->N; a.num_seqs = d->num_seqs;
    a.xb = d->x_stride_b; a.xt = d->x_stride_t;
    a.dtb = d->dt_stride_b; a.dtt = d->dt_stride_t;
    a.bb = d->b_stride_b; a.bt = d->b_stride_t;
    a.cb = d->c_stride_b; a.ct = d->c_stride_t;
    a.h0_f32 = d->initial_state_dtype == KDA_FP32;
    a.ht_f32 = d->final_state_dtype == KDA_FP32;
    a.launch_cap = d->launch_piece;
    return KDA_OK;
}

size_t ssm_state_bytes(const kda_ssm_desc_t *d, int32_t dtype) {
    return (size_t)d->num_seqs * (size_t)d->H * (size_t)(d->P * d->N) * width(dtype);
}
size_t ssm_out_bytes(const kda_ssm_desc_t *d) { return (size_t)(d->B * d->T) * (size_t)(d->H * d->P) * 2; }
void ssm_reads(Memory &m, const void *x, const void *dt, const void *Bm, const void *Cm, const float *A_log,
               const float *dt_bias, const float *D, const void *h0, const int64_t *cu, const kda_ssm_desc_t *d) {
    m.read(x, extent(d->B, d->x_stride_b, d->T, d->x_stride_t, d->H * d->P, 2));
    m.read(dt, extent(d->B, d->dt_stride_b, d->T, d->dt_stride_t, d->H, 2));
    m.read(Bm, extent(d->B, d->b_stride_b, d->T, d->b_stride_t, d->G * d->N, 2));
    m.read(Cm, extent(d->B, d->c_stride_b, d->T, d->c_stride_t, d->G * d->N, 2));
    for (const float *p : {A_log, dt_bias, D}) m.read(p, (size_t)d->H * 4);
    m.read(h0, ssm_state_bytes(d, d->initial_state_dtype));
    m.read(cu, (size_t)(d->num_seqs + 1) * 8);
}

// How a call's sequences are cut into pieces, and its workspace.
struct SsmPlan {
    int64_t cps, pps;                   // chunks / pieces per sequence (not packed)
    int64_t pieces, chunks, slots;      // in all (bounds when packed); slots: pieces of sequences with several
    int pc;                             // chunks per piece
    size_t off_piece, off_chunk, off_slot, off_state, off_decay, total;
};

// Workgroups a launch should have: the two that fit each of the 256 CUs, at once
// and for equal pieces in one round (8192 tokens x 64 heads: 122 us, with two rounds
// 128 us, with a round and a half 131 us).  Under kFewPieces pieces per sequence, two
// rounds: the first pass leaves out the last piece, and one of few leaves CUs idle
// (6 x 4000 tokens x 40 heads: 215 us, with one 219 us).  The pieces of several packed
// sequences are uneven, and take two rounds as well (32768 tokens in 17 sequences: 478
// us, with one 479 us, with three 465 us).
// Fewer than kMinPiece chunks per piece would leave a piece's state (32 KiB of fp32
// per 64 channels and 128 entries) larger than its tokens.
constexpr int64_t kGroups = 512;
constexpr int64_t kMinPiece = 4, kFewPieces = 4;

kda_status_t plan_ssm(const kda_ssm_desc_t *d, bool packed, SsmPlan &p) {
    const int64_t units = d->H * (d->P / 64);
    p = SsmPlan{};
    p.cps = packed ? 0 : (d->T + 63) / 64;
    const bool several = packed && d->num_seqs > 1;
    const int64_t top = several ? d->T / 64 + 1 : (d->T + 63) / 64;  // chunks of the longest sequence
    int64_t pc = d->piece_chunks;
    if (pc == 0) {
        if (several) {
            pc = (top * units + 2 * kGroups - 1) / (2 * kGroups);
        } else {                             // chains that fill the GPU by themselves are not cut
            int64_t pieces = kGroups / std::max<int64_t>(d->B * units, 1);
            if (pieces > 1 && pieces < kFewPieces) pieces *= 2;
            pc = pieces > 1 ? (top + pieces - 1) / pieces : top;
        }
        if (pc < kMinPiece) pc = kMinPiece;
    }
    if (pc > top) pc = top;
    if (pc < 1) pc = 1;
    p.chunks = packed ? d->T / 64 + d->num_seqs : d->B * p.cps;
    p.pps = packed ? 0 : (p.cps + pc - 1) / pc;
    p.pieces = packed ? d->T / (64 * pc) + d->num_seqs : d->B * p.pps;
    // Packed: a sequence of more than 64 pc tokens has under 2 len / (64 pc) pieces.
    p.slots = packed ? std::min(p.pieces, d->T / (32 * pc)) : p.pps > 1 ? p.pieces : 0;
    p.pc = (int)pc;
    // the tables count in 32 bits, and no product of a workspace's sizes passes 63
    if (p.pieces > kMaxSeqs || p.chunks > kMaxSeqs || p.chunks > kMaxTokens / d->H) return KDA_ERR_SHAPE;
    size_t o = 0;
    if (packed) {
        p.off_piece = o; o = align_up(o + (size_t)(d->num_seqs + 1) * 4, 256);
        p.off_chunk = o; o = align_up(o + (size_t)(d->num_seqs + 1) * 4, 256);
        p.off_slot = o; o = align_up(o + (size_t)(d->num_seqs + 1) * 4, 256);
    }
    p.off_state = o; o = align_up(o + (size_t)p.slots * (size_t)d->H * (size_t)(d->P * d->N) * 4, 256);
    p.off_decay = o; o = align_up(o + (size_t)p.slots * (size_t)d->H * 4, 256);
    p.total = o;
    return KDA_OK;
}

// The gradient's workspace: the forward's, then the states and the sums.
struct SsmBwdPlan {
    SsmPlan p;
    int share, shares;                  // heads of a group per workgroup, workgroups per chunk and group
    size_t off_hs, off_ds, off_psum, off_part, total;
};

// With few chunks the heads of a group are shared out among workgroups, of which one
// fits each CU, and the shares' dB and dC added up.  In units of a workgroup's time
// for one head and 64 channels (7 us at 128 entries), a round costs its heads and
// about one more to begin, and adding up about one per 256 shares (128 chunks x 64
// heads: 2 shares 510 us, 4 522 us, 8 544 us).
int64_t grad_shares(int64_t groups, int64_t heads, int64_t blocks) {
    constexpr int64_t kCus = 256, kMost = 64;
    int64_t best = 1, least = INT64_MAX;
    for (int64_t s = 1; s <= heads && s <= kMost; ++s) {
        const int64_t share = (heads + s - 1) / s, all = groups * s;
        const int64_t cost = (all + kCus - 1) / kCus * (share * blocks + 1) + (s > 1 ? (all + kCus - 1) / kCus : 0);
        if (cost < least) {
            least = cost;
            best = s;
        }
    }
    return best;
}

kda_status_t plan_ssm_bwd(const kda_ssm_desc_t *d, bool packed, SsmBwdPlan &b) {
    const kda_status_t st = plan_ssm(d, packed, b.p);
    if (st != KDA_OK) return st;
    const int64_t heads = d->H / d->G, chunks = b.p.chunks, groups = chunks * d->G;
    const int64_t shares = grad_shares(groups, heads, d->P / 64);
    const int64_t share = (heads + shares - 1) / shares;
    b.share = (int)share;
    b.shares = (int)((heads + share - 1) / share);
    const size_t states = (size_t)chunks * (size_t)d->H * (size_t)(d->P * d->N) * 4;
    size_t o = b.p.total;
    b.off_hs = o; o = align_up(o + states, 256);
    b.off_ds = o; o = align_up(o + states, 256);
    b.off_psum = o; o = align_up(o + (size_t)chunks * (size_t)d->H * 16, 256);
    b.off_part = o;
    if (b.shares > 1) o = align_up(o + 2 * (size_t)b.shares * (size_t)groups * (size_t)(64 * d->N) * 4, 256);
    b.total = o;
    return KDA_OK;
}

// The larger of the packed and unpacked needs, where both are possible.
template <typename F>
int64_t over_plans(const kda_ssm_desc_t *d, F f) {
    int64_t best = -1;
    if (!d) return best;
    for (bool packed : {false, true}) {
        SsmPlan p;
        if (check_ssm(d, packed) != KDA_OK || plan_ssm(d, packed, p) != KDA_OK) continue;
        const int64_t v = f(p);
        best = v > best ? v : best;
    }
    return best;
}

SsmChainArgs chain_args(const SsmArgs &a, const SsmPlan &p, const Workspace &ws) {
    SsmChainArgs c{};
    c.x = a.x; c.k = a.Bm; c.c = a.Cm; c.dt = a.dt;
    c.xb = a.xb; c.xt = a.xt; c.kb = a.bb; c.kt = a.bt; c.cb = a.cb; c.ct = a.ct; c.dtb = a.dtb; c.dtt = a.dtt;
    c.A_log = a.A_log; c.dt_bias = a.dt_bias; c.D = a.D;
    c.cu = a.cu;
    c.launch_cap = a.launch_cap;
    c.T = a.T; c.H = a.H; c.P = a.P; c.G = a.G; c.seqs = a.num_seqs;
    c.pieces = p.pieces; c.chunks = p.chunks; c.slots = p.slots; c.pps = p.pps; c.cps = p.cps; c.pc = p.pc;
    if (a.cu) {
        c.piece_off = reinterpret_cast<const int32_t *>(ws.at(p.off_piece));
        c.chunk_off = reinterpret_cast<const int32_t *>(ws.at(p.off_chunk));
        c.slot_off = reinterpret_cast<const int32_t *>(ws.at(p.off_slot));
    }
    if (p.slots > 0) {
        c.state = reinterpret_cast<float *>(ws.at(p.off_state));
        c.decay = reinterpret_cast<float *>(ws.at(p.off_decay));
    }
    return c;
}

hipError_t launch_table(const SsmArgs &a, const SsmPlan &p, const Workspace &ws, hipStream_t s) {
    if (!a.cu) return hipSuccess;
    return kda_launch_ssm_table({a.cu, a.num_seqs, a.T, p.pc, p.pieces, p.chunks, p.slots,
                                 reinterpret_cast<int32_t *>(ws.at(p.off_piece)), reinterpret_cast<int32_t *>(ws.at(p.off_chunk)),
                                 reinterpret_cast<int32_t *>(ws.at(p.off_slot))}, s);
}

// The states entering the pieces, and the final states of empty sequences.
// Nothing to do for sequences of one piece each.
hipError_t launch_entering(const SsmChainArgs &c, int N, bool reverse, hipStream_t s) {
    if (!c.cu && c.pps == 1) return hipSuccess;
    hipError_t e = hipSuccess;
    if (c.slots > 0) e = kda_launch_ssm_pieces(c, N, reverse, s);
    if (e == hipSuccess) e = kda_launch_ssm_scan(c, N, reverse, s);
    return e;
}

}  // namespace

extern "C" kda_status_t kda_rmsnorm_fwd(const void *x, const void *residual, const void *weight, void *residual_out,
                                        void *out, const kda_rmsnorm_desc_t *desc, hipStream_t stream) {
    return norm_impl(x, residual, weight, residual_out, out, nullptr, 0, desc, stream);
}

extern "C" kda_status_t kda_rmsnorm_quant(const void *x, const void *residual, const void *weight,
                                          void *residual_out, void *out_q, float *scales,
                                          const kda_rmsnorm_desc_t *desc, hipStream_t stream) {
    if (desc && desc->group != 0 && desc->group != 128) return KDA_ERR_PARAM;
    return norm_impl(x, residual, weight, residual_out, out_q, scales, 1, desc, stream);
}

namespace {
struct NormBwdLayout {
    size_t off_rstd, off_part, total;
    int64_t parts;
};
NormBwdLayout norm_bwd_layout(const kda_rmsnorm_desc_t *d) {
    NormBwdLayout l{};
    l.parts = kda_rmsnorm_parts(d->rows, d->D);
    l.off_rstd = 0;
    l.off_part = align_up((size_t)d->rows * 4, 256);
    l.total = align_up(l.off_part + (size_t)l.parts * (size_t)d->D * 4, 256);
    return l;
}
}  // namespace

extern "C" size_t kda_rmsnorm_bwd_workspace_size(const kda_rmsnorm_desc_t *desc) {
    if (!desc || desc->rows < 0 || desc->D < 1 || desc->rows > kMaxTokens || desc->D > kMaxColumns) return 0;
    return norm_bwd_layout(desc).total;
}

extern "C" kda_status_t kda_rmsnorm_bwd(const void *h, const void *weight, const void *d_out,
                                        const void *d_residual_out, void *dx, float *dresidual, float *dweight,
                                        const kda_rmsnorm_desc_t *desc, hipStream_t stream) {
    if (!desc || !weight || !dweight) return KDA_ERR_NULL;
    kda_status_t st = check_norm(desc);
    if (st != KDA_OK) return st;
    if (desc->rows > 0 && (!h || !d_out || !dx)) return KDA_ERR_NULL;
    if (!dtype_ok(desc->residual_dtype)) return KDA_ERR_DTYPE;
    if (dresidual && desc->residual_dtype != KDA_FP32) return KDA_ERR_DTYPE;
    if (!stride_ok(desc->d_out_stride) || (d_residual_out && !stride_ok(desc->d_residual_stride))) return KDA_ERR_SHAPE;
    const size_t hw = width(desc->residual_dtype);
    if (!aligned(h, hw) || !aligned(d_residual_out, hw) || !aligned(d_out, 2) || !aligned(dx, 2) || !aligned(dresidual, 4) ||
        !aligned(dweight, 4) || !aligned(weight, width(desc->weight_dtype)))
        return KDA_ERR_ALIGN;
    const NormBwdLayout l = norm_bwd_layout(desc);
    const size_t n = (size_t)desc->rows * (size_t)desc->D;
    Memory m;
    m.read(h, extent(1, 0, desc->rows, desc->x_stride, desc->D, hw));
    m.read(weight, (size_t)desc->D * width(desc->weight_dtype));
    m.read(d_out, extent(1, 0, desc->rows, desc->d_out_stride, desc->D, 2));
    m.read(d_residual_out, extent(1, 0, desc->rows, desc->d_residual_stride, desc->D, hw));
    m.write(dx, n * 2);
    m.write(dresidual, n * 4);
    m.write(dweight, (size_t)desc->D * 4);
    m.write(desc->workspace, l.total);
    if (m.clash()) return KDA_ERR_OVERLAP;
    Workspace ws(desc->workspace, desc->workspace_bytes, l.total, stream);
    if (ws.status() != KDA_OK) return ws.status();
    NormBwdArgs a{};
    a.h = h; a.w = weight; a.dy = static_cast<const uint16_t *>(d_out); a.dres = d_residual_out;
    a.dx = static_cast<uint16_t *>(dx); a.dresidual = dresidual; a.dw = dweight;
    a.rstd = reinterpret_cast<float *>(ws.at(l.off_rstd));
    a.part = reinterpret_cast<float *>(ws.at(l.off_part));
    a.rows = desc->rows; a.D = desc->D; a.hs = desc->x_stride; a.ds = desc->d_out_stride;
    a.rs = desc->d_residual_stride; a.parts = l.parts;
    a.eps = desc->eps;
    a.h_f32 = desc->residual_dtype == KDA_FP32;
    a.w_f32 = desc->weight_dtype == KDA_FP32;
    return of_hip(kda_launch_rmsnorm_bwd(a, stream));
}

extern "C" kda_status_t kda_conv_fwd(const void *x, const void *weight, const void *bias, const void *initial_state,
                                     void *final_state, const int64_t *cu_seqlens, void *out,
                                     const kda_conv_desc_t *desc, hipStream_t stream) {
    ConvArgs a;
    kda_status_t st = conv_args(x, weight, bias, initial_state, final_state, cu_seqlens, desc, a);
    if (st != KDA_OK) return st;
    if (desc->T > 0 && !out) return KDA_ERR_NULL;
    if (!aligned(out, 2)) return KDA_ERR_ALIGN;
    Memory m;
    conv_reads(m, x, weight, bias, initial_state, cu_seqlens, desc);
    m.write(out, conv_token_bytes(desc));
    m.write(final_state, conv_state_bytes(desc, desc->final_state_dtype), initial_state);
    if (m.clash()) return KDA_ERR_OVERLAP;
    st = validate_cu(cu_seqlens, desc->num_seqs, desc->T, stream);
    if (st != KDA_OK) return st;
    a.ht = final_state;
    a.out = static_cast<uint16_t *>(out);
    return of_hip(kda_launch_conv(a, (int)desc->W, stream));
}

extern "C" kda_status_t kda_conv_decode(const void *x, const void *weight, const void *bias,
                                        const void *initial_state, void *final_state, void *out,
                                        const kda_conv_desc_t *desc, hipStream_t stream) {
    ConvArgs a;
    const kda_status_t st = conv_args(x, weight, bias, initial_state, final_state, nullptr, desc, a);
    if (st != KDA_OK) return st;
    if (desc->T != 1) return KDA_ERR_SHAPE;
    if (!out || !final_state) return KDA_ERR_NULL;
    if (!aligned(out, 2)) return KDA_ERR_ALIGN;
    Memory m;
    conv_reads(m, x, weight, bias, initial_state, nullptr, desc);
    m.write(out, conv_token_bytes(desc));
    m.write(final_state, conv_state_bytes(desc, desc->final_state_dtype), initial_state);
    if (m.clash()) return KDA_ERR_OVERLAP;
    a.ht = final_state;
    a.out = static_cast<uint16_t *>(out);
    return of_hip(kda_launch_conv_decode(a, (int)desc->W, stream));
}

extern "C" size_t kda_conv_bwd_workspace_size(const kda_conv_desc_t *desc) {
    if (!desc || (check_conv(desc, false) != KDA_OK && check_conv(desc, true) != KDA_OK)) return 0;
    return align_up((size_t)kda_conv_parts(desc->B, desc->T, desc->D) * (size_t)(desc->W + 1) * (size_t)desc->D * 4, 256);
}

extern "C" kda_status_t kda_conv_bwd(const void *x, const void *weight, const void *bias, const void *initial_state,
                                     const int64_t *cu_seqlens, const void *d_out, const void *d_final_state,
                                     void *dx, float *dweight, float *dbias, float *d_initial_state,
                                     const kda_conv_desc_t *desc, hipStream_t stream) {
    ConvArgs a;
    kda_status_t st = conv_args(x, weight, bias, initial_state, d_final_state, cu_seqlens, desc, a);
    if (st != KDA_OK) return st;
    if (!dweight || (desc->T > 0 && (!d_out || !dx))) return KDA_ERR_NULL;
    if (!stride_ok(desc->d_out_stride_b) || !stride_ok(desc->d_out_stride_t)) return KDA_ERR_SHAPE;
    if (!aligned(d_out, 2) || !aligned(dx, 2) || !aligned(dweight, 4) || !aligned(dbias, 4) || !aligned(d_initial_state, 4))
        return KDA_ERR_ALIGN;
    Memory m;
    conv_reads(m, x, weight, bias, initial_state, cu_seqlens, desc);
    m.read(d_out, extent(desc->B, desc->d_out_stride_b, desc->T, desc->d_out_stride_t, desc->D, 2));
    m.read(d_final_state, conv_state_bytes(desc, desc->final_state_dtype));
    m.write(dx, conv_token_bytes(desc));
    m.write(dweight, (size_t)(desc->D * desc->W) * 4);
    m.write(dbias, (size_t)desc->D * 4);
    m.write(d_initial_state, conv_state_bytes(desc, KDA_FP32));
    m.write(desc->workspace, kda_conv_bwd_workspace_size(desc));
    if (m.clash()) return KDA_ERR_OVERLAP;
    st = validate_cu(cu_seqlens, desc->num_seqs, desc->T, stream);
    if (st != KDA_OK) return st;
    Workspace ws(desc->workspace, desc->workspace_bytes, kda_conv_bwd_workspace_size(desc), stream);
    if (ws.status() != KDA_OK) return ws.status();
    a.dy = static_cast<const uint16_t *>(d_out);
    a.db_ = desc->d_out_stride_b; a.dt_ = desc->d_out_stride_t;
    a.dht = d_final_state;
    a.dx = static_cast<uint16_t *>(dx);
    a.dw = dweight; a.dbias = dbias; a.dh0 = d_initial_state;
    a.part = reinterpret_cast<float *>(ws.at(0));
    a.parts = kda_conv_parts(desc->B, desc->T, desc->D);
    return of_hip(kda_launch_conv_bwd(a, (int)desc->W, stream));
}

extern "C" kda_status_t kda_ssm_decode(const void *x, const void *dt, const void *Bm, const void *Cm,
                                       const float *A_log, const float *dt_bias, const float *D,
                                       const void *initial_state, void *final_state, void *out,
                                       const kda_ssm_desc_t *desc, hipStream_t stream) {
    SsmArgs a;
    const kda_status_t st = ssm_args(x, dt, Bm, Cm, A_log, dt_bias, D, initial_state, final_state, nullptr, desc, a);
    if (st != KDA_OK) return st;
    if (desc->T != 1) return KDA_ERR_SHAPE;
    if (!out || !final_state) return KDA_ERR_NULL;
    if (!aligned(out, 16)) return KDA_ERR_ALIGN;
    Memory m;
    ssm_reads(m, x, dt, Bm, Cm, A_log, dt_bias, D, initial_state, nullptr, desc);
    m.write(out, ssm_out_bytes(desc));
    m.write(final_state, ssm_state_bytes(desc, desc->final_state_dtype), initial_state);
    if (m.clash()) return KDA_ERR_OVERLAP;
    a.ht = final_state;
    a.out = static_cast<uint16_t *>(out);
    return of_hip(kda_launch_ssm_decode(a, stream));
}

extern "C" size_t kda_ssm_fwd_workspace_size(const kda_ssm_desc_t *desc) {
    const int64_t n = over_plans(desc, [](const SsmPlan &p) { return (int64_t)p.total; });
    return n > 0 ? (size_t)n : 0;
}

extern "C" int64_t kda_ssm_piece_chunks(const kda_ssm_desc_t *desc) {
    SsmPlan p;
    const bool packed = desc && desc->num_seqs != desc->B;
    if (!desc || check_ssm(desc, packed) != KDA_OK || plan_ssm(desc, packed, p) != KDA_OK) return -1;
    return p.pc;
}

extern "C" kda_status_t kda_ssm_fwd(const void *x, const void *dt, const void *Bm, const void *Cm, const float *A_log,
                                    const float *dt_bias, const float *D, const void *initial_state,
                                    void *final_state, const int64_t *cu_seqlens, void *out,
                                    const kda_ssm_desc_t *desc, hipStream_t stream) {
    SsmArgs a;
    kda_status_t st = ssm_args(x, dt, Bm, Cm, A_log, dt_bias, D, initial_state, final_state, cu_seqlens, desc, a);
    if (st != KDA_OK) return st;
    if (desc->T > 0 && !out) return KDA_ERR_NULL;
    if (!aligned(out, 16)) return KDA_ERR_ALIGN;
    SsmPlan p;
    st = plan_ssm(desc, cu_seqlens != nullptr, p);
    if (st != KDA_OK) return st;
    Memory m;
    ssm_reads(m, x, dt, Bm, Cm, A_log, dt_bias, D, initial_state, cu_seqlens, desc);
    m.write(out, ssm_out_bytes(desc));
    m.write(final_state, ssm_state_bytes(desc, desc->final_state_dtype), initial_state);
    m.write(desc->workspace, p.total);
    if (m.clash()) return KDA_ERR_OVERLAP;
    st = validate_cu(cu_seqlens, desc->num_seqs, desc->T, stream);
    if (st != KDA_OK) return st;
    Workspace ws(desc->workspace, desc->workspace_bytes, p.total, stream);
    if (ws.status() != KDA_OK) return ws.status();
    SsmChainArgs c = chain_args(a, p, ws);
    c.h0 = initial_state; c.h0_f32 = a.h0_f32;
    c.ht = final_state; c.ht_f32 = a.ht_f32;
    c.out = static_cast<uint16_t *>(out);
    const int N = (int)desc->N;
    hipError_t e = launch_table(a, p, ws, stream);
    if (e == hipSuccess) e = launch_entering(c, N, false, stream);
    if (e == hipSuccess && desc->T > 0) e = kda_launch_ssm_chain(c, N, stream);
    return of_hip(e);
}

extern "C" size_t kda_ssm_bwd_workspace_size(const kda_ssm_desc_t *desc) {
    size_t best = 0;
    if (!desc) return 0;
    for (bool packed : {false, true}) {
        SsmBwdPlan b;
        if (check_ssm(desc, packed) != KDA_OK || plan_ssm_bwd(desc, packed, b) != KDA_OK) continue;
        best = b.total > best ? b.total : best;
    }
    return best;
}

extern "C" kda_status_t kda_ssm_bwd(const void *x, const void *dt, const void *Bm, const void *Cm, const float *A_log,
                                    const float *dt_bias, const float *D, const void *initial_state,
                                    const int64_t *cu_seqlens, const void *d_out, const void *d_final_state, void *dx,
                                    void *ddt, void *dB, void *dC, float *dA_log, float *ddt_bias, float *dD,
                                    float *d_initial_state, const kda_ssm_desc_t *desc, hipStream_t stream) {
    SsmArgs a;
    kda_status_t st = ssm_args(x, dt, Bm, Cm, A_log, dt_bias, D, initial_state, d_final_state, cu_seqlens, desc, a);
    if (st != KDA_OK) return st;
    if (!dA_log || (desc->T > 0 && (!d_out || !dx || !ddt || !dB || !dC))) return KDA_ERR_NULL;
    if (!stride_ok(desc->d_out_stride_b) || !stride_ok(desc->d_out_stride_t) || desc->d_out_stride_t >= kMaxTokenStride)
        return KDA_ERR_SHAPE;
    if (desc->d_out_stride_b % 8 || desc->d_out_stride_t % 8 || !aligned(d_out, 16) || !aligned(dx, 16) || !aligned(ddt, 2) ||
        !aligned(dB, 16) || !aligned(dC, 16) || !aligned(dA_log, 4) || !aligned(ddt_bias, 4) || !aligned(dD, 4) ||
        !aligned(d_initial_state, 16))
        return KDA_ERR_ALIGN;
    SsmBwdPlan b;
    st = plan_ssm_bwd(desc, cu_seqlens != nullptr, b);
    if (st != KDA_OK) return st;
    const size_t tokens = (size_t)(desc->B * desc->T), bc = tokens * (size_t)(desc->G * desc->N) * 2;
    Memory m;
    ssm_reads(m, x, dt, Bm, Cm, A_log, dt_bias, D, initial_state, cu_seqlens, desc);
    m.read(d_out, extent(desc->B, desc->d_out_stride_b, desc->T, desc->d_out_stride_t, desc->H * desc->P, 2));
    m.read(d_final_state, ssm_state_bytes(desc, desc->final_state_dtype));
    m.write(dx, ssm_out_bytes(desc));
    m.write(ddt, tokens * (size_t)desc->H * 2);
    m.write(dB, bc);
    m.write(dC, bc);
    for (float *q : {dA_log, ddt_bias, dD}) m.write(q, (size_t)desc->H * 4);
    m.write(d_initial_state, ssm_state_bytes(desc, KDA_FP32));
    m.write(desc->workspace, b.total);
    if (m.clash()) return KDA_ERR_OVERLAP;
    st = validate_cu(cu_seqlens, desc->num_seqs, desc->T, stream);
    if (st != KDA_OK) return st;
    Workspace ws(desc->workspace, desc->workspace_bytes, b.total, stream);
    if (ws.status() != KDA_OK) return ws.status();

    const int N = (int)desc->N;
    SsmChainArgs f = chain_args(a, b.p, ws);     // the states
    f.h0 = initial_state; f.h0_f32 = a.h0_f32;
    f.save = reinterpret_cast<float *>(ws.at(b.off_hs));
    SsmChainArgs r = f;                          // their gradients: from d_out and C, last token first
    r.x = static_cast<const uint16_t *>(d_out); r.xb = desc->d_out_stride_b; r.xt = desc->d_out_stride_t;
    r.k = a.Cm; r.kb = a.cb; r.kt = a.ct;
    r.h0 = d_final_state; r.h0_f32 = a.ht_f32;
    r.ht = d_initial_state; r.ht_f32 = 1;
    r.save = reinterpret_cast<float *>(ws.at(b.off_ds));
    SsmGradArgs g{};
    g.x = a.x; g.Bm = a.Bm; g.Cm = a.Cm; g.dt = a.dt; g.dy = static_cast<const uint16_t *>(d_out);
    g.xb = a.xb; g.xt = a.xt; g.bb = a.bb; g.bt = a.bt; g.cb = a.cb; g.ct = a.ct; g.dtb = a.dtb; g.dtt = a.dtt;
    g.yb = desc->d_out_stride_b; g.yt = desc->d_out_stride_t;
    g.A_log = A_log; g.dt_bias = dt_bias; g.D = D;
    g.launch_cap = a.launch_cap;
    g.cu = cu_seqlens; g.chunk_off = f.chunk_off;
    g.T = a.T; g.H = a.H; g.P = a.P; g.G = a.G; g.seqs = a.num_seqs;
    g.chunks = b.p.chunks; g.cps = b.p.cps;
    g.share = b.share; g.shares = b.shares;
    g.hs = f.save; g.ds = r.save;
    g.dx = static_cast<uint16_t *>(dx); g.ddt = static_cast<uint16_t *>(ddt);
    g.dB = static_cast<uint16_t *>(dB); g.dC = static_cast<uint16_t *>(dC);
    g.psum = reinterpret_cast<float *>(ws.at(b.off_psum));
    g.part = reinterpret_cast<float *>(ws.at(b.off_part));
    g.dA_log = dA_log; g.ddt_bias = ddt_bias; g.dD = dD;

    hipError_t e = launch_table(a, b.p, ws, stream);
    if (e == hipSuccess) e = launch_entering(f, N, false, stream);
    if (e == hipSuccess && desc->T > 0) e = kda_launch_ssm_save(f, N, false, stream);
    if (e == hipSuccess) e = launch_entering(r, N, true, stream);
    if (e == hipSuccess && desc->T > 0) e = kda_launch_ssm_save(r, N, true, stream);
    if (e == hipSuccess) e = kda_launch_ssm_grad(g, N, stream);
    return of_hip(e);
}
