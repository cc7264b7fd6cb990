// delta_ranges.cpp -- the extents that the gated delta rule's kernels give to the
// hardware's range checks, taken on the host: no range may reach past its tensor, whatever
// a kernel reads at a row's last columns.  Host only.
#include <stdint.h>
#include <stdio.h>

#include "../../implicit_gemm_conv_amd/csrc/delta_params.h"

using namespace convdelta;

namespace {

long wrong = 0;

void expect(bool ok, const char* what, int64_t got, int64_t want) {
  if (ok) return;
  ++wrong;
  fprintf(stderr, "%s: %lld, expected %lld\n", what, (long long)got, (long long)want);
}

// Rows of y, x and v's gradient of every chunk and head: they lie in the tensor, hold all of the head's columns, and those of
// the last head's last row end where the tensor does.
void dense(int b, int t, int hv, int dv, int elem) {
  DeltaArgs a{};
  a.b = b, a.t = t, a.hv = hv, a.dv = dv;
  a.chunks = (t + kChunk - 1) / kChunk;
  const int64_t all = (int64_t)b * t * hv * dv * elem;
  for (int i = 0; i < b; ++i)
    for (int h = 0; h < hv; ++h)
      for (int c = 0; c < a.chunks; ++c) {
        const Span s = dense_rows(a, i, h, c, elem);
        const int rows = c + 1 < a.chunks ? kChunk : t - c * kChunk;
        const int64_t first = (((int64_t)i * t + c * kChunk) * hv + h) * dv * elem;
        expect(s.at == first, "a range's first byte", s.at, first);
        const int64_t last = first + ((int64_t)(rows - 1) * hv + 1) * dv * elem;
        expect(s.at + s.bytes == last, "a range's end", s.at + s.bytes, last);
        expect(s.at + s.bytes <= all, "a range past its tensor", s.at + s.bytes, all);
      }
}

// 64 rows of the copies of q and k, whatever the number of heads: offsets below 2^31, where the offset that marks what is
// not there lies, and every element of the copy its own.
void packed(int b, int t, int hk, int dkp, int elem) {
  const Heads h = packed_rows(nullptr, t, hk, dkp);
  const int64_t far = (63 * h.st + dkp) * elem;
  expect(far < (int64_t)1 << 31, "64 rows of a copy", far, (int64_t)1 << 31);
  const int64_t last = (b - 1) * h.sb + (t - 1) * h.st + (hk - 1) * h.sh + dkp, all = (int64_t)b * t * hk * dkp;
  expect(last == all, "a copy's last element", last, all);
  expect(h.st >= dkp && h.sh == t * h.st && h.sb == hk * h.sh, "a copy's strides", h.st, dkp);
}

}  // namespace

int main() {
  for (const int elem : {2, 4})
    for (const int b : {1, 3})
      for (const int t : {1, 64, 1000})
        for (const int hk : {1, 7, 1 << 17, 1 << 18, (1 << 21) - 1})
          for (const int dkp : {8, 72, 120, 128}) packed(b, t, hk, dkp, elem);
  for (const int elem : {2, 4})
    for (const int b : {1, 2})
      for (const int t : {1, 2, 63, 64, 65, 130})
        for (const int hv : {1, 2, 5})
          for (const int dv : {1, 3, 4, 33, 130}) dense(b, t, hv, dv, elem);
  printf("%ld wrong ranges\n", wrong);
  return wrong != 0;
}
