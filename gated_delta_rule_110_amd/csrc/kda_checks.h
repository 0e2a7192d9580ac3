// kda_checks.h -- what the C ABI's host sides have in common: limits, argument
// checks, workspaces.
#pragma once
#include <stdlib.h>
#include <new>
#include "kda.h"

namespace kda {

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool dtype_ok(int32_t d) { return d == KDA_BF16 || d == KDA_FP32; }
inline size_t width(int32_t d) { return d == KDA_FP32 ? 4 : 2; }

// Sizes beyond these are refused, so that no product of a call's sizes passes
// 63 bits (rows and columns) or a grid's 2^31 - 1 workgroups.
constexpr int64_t kMaxTokens = int64_t(1) << 40;
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxTokenStride = int64_t(1) << 24;
constexpr int64_t kMaxSeqs = 0x7fffffff;

inline bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }

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
inline size_t extent(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t inner, size_t w) {
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

inline kda_status_t of_hip(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

// KDA_VALIDATE=1: the contents of cu_seqlens, read back to the host.
inline kda_status_t validate_cu(const int64_t *cu, int64_t N, int64_t T, hipStream_t stream) {
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

}  // namespace kda
