// seq_buffers.h -- what the C entry points beside the convolution share on the
// host: element sizes, the check of a call's buffers, the launch's answer.
#pragma once

#include "../../include/convseq.h"

#include <stdint.h>

#include "conv_params.h"
#include "seq_params.h"

namespace convseq {

inline int elem_bytes(int dtype) { return dtype == CONVFWD_F32 ? 4 : 2; }
inline int launched(hipError_t e) { return e == hipSuccess ? CONVFWD_OK : CONVFWD_ERR_LAUNCH; }

// The buffers of one call: checks each as it is added (present, aligned,
// strides) and that no output overlaps another buffer.
class Buffers {
 public:
  // `need`: the buffer has to be given; `bytes` 0: it is not accessed.
  void in(const void* p, int64_t bytes, int align, bool need = true) { add(p, bytes, align, need, false); }
  void out(const void* p, int64_t bytes, int align, bool need = true) { add(p, bytes, align, need, true); }
  void rows(const convseq_rows* r, int64_t b, int64_t t, int64_t c, int elem, Rows* to) {
    *to = Rows{nullptr, 0, 0};
    if (!r) return fail(CONVFWD_ERR_NULL);
    if (r->batch_stride < 0 || r->row_stride < 0) return fail(CONVFWD_ERR_BAD_DESC);
    // 2^62 bytes is past any address range; keeps the sums below in 64 bits
    const int64_t lim = (int64_t)1 << 62;
    const int64_t nb = b > 1 ? b - 1 : 0, nt = t > 1 ? t - 1 : 0;
    if ((nb && r->batch_stride > lim / 8 / nb) || (nt && r->row_stride > lim / 8 / nt))
      return fail(CONVFWD_ERR_TOO_LARGE);
    const bool empty = b == 0 || t == 0;
    in(r->data, empty ? 0 : (nb * r->batch_stride + nt * r->row_stride + c) * elem, elem);
    *to = Rows{r->data, r->batch_stride, r->row_stride};
  }
  // A (B, T, C) tensor in 8 bits, read or written.
  void kept(const convseq_kept* k, int64_t b, int64_t t, int64_t c, bool write, Kept* to) {
    *to = Kept{nullptr, nullptr};
    if (!k) return;
    const int64_t e = b * ((t + kGroup - 1) / kGroup) * c;
    add(k->q, e * kGroup, kGroup, true, write);
    add(k->e, e, 1, true, write);
    *to = Kept{(int8_t*)k->q, (uint8_t*)k->e};
  }
  int result() const {
    if (rc_ < 0) return rc_;
    for (int i = 0; i < n_; ++i)
      for (int j = 0; j < i; ++j)
        if ((b_[i].out || b_[j].out) && b_[i].lo < b_[j].hi && b_[j].lo < b_[i].hi) return CONVFWD_ERR_ALIAS;
    return CONVFWD_OK;
  }

 private:
  void fail(int rc) {
    if (rc_ == CONVFWD_OK) rc_ = rc;
  }
  void add(const void* p, int64_t bytes, int align, bool need, bool out) {
    if (!p) {
      if (need && bytes > 0) fail(CONVFWD_ERR_NULL);
      return;
    }
    if ((uintptr_t)p % align) return fail(CONVFWD_ERR_MISALIGNED);
    if (bytes <= 0) return;
    b_[n_++] = Range{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, out};
  }
  struct Range {
    uintptr_t lo, hi;
    bool out;
  };
  Range b_[24];  // the longest call adds 17
  int n_ = 0, rc_ = CONVFWD_OK;
};

}  // namespace convseq
