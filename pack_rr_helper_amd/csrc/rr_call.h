// rr_call.h -- what the host layers of the operators share: checks of a call's
// arguments and buffers, the division of a workspace, and the launches of a call.
#pragma once

#include "rr_loss.h"

namespace rr {
namespace {

inline int64_t elem_size(int dtype) { return dtype == RR_F32 ? 4 : 2; }
inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

inline rr_status check_dtype(int dtype)
{
    if (dtype != RR_F32 && dtype != RR_BF16)
        return set_error(RR_EINVAL, "unknown dtype %d", dtype);
    return RR_OK;
}

inline rr_status check_workspace(int64_t have, int64_t need)
{
    if (have < need)
        return set_error(RR_EINVAL, "workspace of %lld bytes, needs %lld", (long long)have, (long long)need);
    return RR_OK;
}

// The buffers of one call: each checked for null and alignment, the written
// ones against every other.
class Buffers {
public:
    Buffers &in(const void *p, int64_t bytes, int64_t align, const char *what) { return add(p, bytes, align, what, false); }
    Buffers &out(const void *p, int64_t bytes, int64_t align, const char *what) { return add(p, bytes, align, what, true); }

    rr_status check()
    {
        if (st_ != RR_OK)
            return st_;
        for (int i = 0; i < n_; ++i)
            for (int j = 0; j < i; ++j)
                if ((b_[i].written || b_[j].written) && b_[i].lo < b_[j].hi && b_[j].lo < b_[i].hi)
                    return set_error(RR_EALIAS, "%s overlaps %s", b_[i].what, b_[j].what);
        return RR_OK;
    }

private:
    struct Buf {
        uintptr_t lo, hi;
        const char *what;
        bool written;
    };
    Buffers &add(const void *p, int64_t bytes, int64_t align, const char *what, bool written)
    {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        if (st_ != RR_OK || bytes <= 0)
            return *this;
        if (!p)
            st_ = set_error(RR_EINVAL, "%s is null", what);
        else if (lo % uintptr_t(align))
            st_ = set_error(RR_EINVAL, "%s=%p is not aligned to %lld bytes", what, p, (long long)align);
        else
            b_[n_++] = Buf{lo, lo + uintptr_t(bytes), what, written};
        return *this;
    }
    Buf b_[2 * RR_MAX_SHARDS + 16];
    int n_ = 0;
    rr_status st_ = RR_OK;
};

// The launches of one call, up to the first that fails.
class Launches {
public:
    explicit Launches(void *stream) : st_(static_cast<hipStream_t>(stream)) {}
    template <typename A>
    void add(hipError_t (*launch)(const Op &, hipStream_t), const A &a)
    {
        if (err_ == hipSuccess)
            err_ = emit_op(Op::make(launch, a), st_);
    }
    rr_status finish() const { return err_ == hipSuccess ? set_ok() : op_failed(err_); }

private:
    hipStream_t st_;
    hipError_t err_ = hipSuccess;
};

// Parts of a workspace, one after the other at 256-byte boundaries.
class Carver {
public:
    explicit Carver(void *base) : base_(static_cast<char *>(base)) {}
    void *take(int64_t bytes)
    {
        void *p = base_ + used_;
        used_ += round_up(bytes, 256);
        return p;
    }
    int64_t used() const { return used_; }

private:
    char *base_;
    int64_t used_ = 0;
};

}  // namespace
}  // namespace rr
