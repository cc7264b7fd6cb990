// seq_fuzz.cpp -- drives the host side of include/convseq.h under sanitizers:
// random (valid and invalid) descriptors, views and buffers through every entry
// point from several threads.  No call launches: each either has something that
// validation refuses, or describes an empty batch.
//
//   seq_fuzz THREADS ROUNDS
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <atomic>
#include <thread>
#include <vector>

#include "../../include/convseq.h"

namespace {

struct Rng {
  uint64_t s;
  uint32_t next() {
    s = s * 6364136223846793005ull + 1442695040888963407ull;
    return (uint32_t)(s >> 33);
  }
  int of(int n) { return (int)(next() % (uint32_t)n); }
};

std::atomic<long> wrong{0};

void expect(bool ok, const char* what, int rc) {
  if (!ok) {
    ++wrong;
    fprintf(stderr, "%s: %d\n", what, rc);
  }
}

// Addresses far apart that nothing reads: validation looks at their values only.
void* at(Rng& r) { return (void*)(((uintptr_t)r.of(64) + 1) << 32); }

void run(int id, int rounds) {
  Rng r{(uint64_t)id * 7919 + 1};
  static const int32_t odd[] = {-2147483647, -1, 0, 1, 2, 15, 16, 17, 64, 1000, 65537, 1 << 22, 1 << 26, 2147483647};
  for (int n = 0; n < rounds; ++n) {
    const auto pick = [&] { return odd[r.of(14)]; };
    convseq_conv_desc c = {pick(), pick(), pick(), r.of(12) - 1, r.of(4) - 1, r.of(5) - 1};
    convseq_scan_desc s = {c.b, c.t, c.c, c.dtype, r.of(3) ? 8.f : -1.f};
    const int64_t cw = convseq_conv_bwd_workspace(&c), fw = convseq_scan_fwd_workspace(&s), bw = convseq_scan_bwd_workspace(&s);
    expect((cw < 0) == (c.b < 0 || c.t < 0 || c.c < 1 || c.k < 1 || c.k > 8 || c.act < 0 || c.act > 1 || c.dtype < 0 ||
                        c.dtype > 2 || cw == CONVFWD_ERR_TOO_LARGE), "conv workspace", (int)cw);
    expect((fw < 0) == (bw < 0) && cw >= -7 && fw >= -7, "scan workspace", (int)fw);
    // something is missing: never launches
    convseq_rows rows = {at(r), (int64_t)r.next() << (r.of(3) * 14), (int64_t)r.next() << (r.of(3) * 14)};
    convseq_kept kept[3] = {{at(r), at(r)}, {at(r), at(r)}, {at(r), nullptr}};
    int rc = convseq_conv_fwd(&c, &rows, nullptr, at(r), at(r), at(r), at(r), at(r), kept, nullptr);
    expect(rc < 0, "conv_fwd without w", rc);
    rc = convseq_conv_bwd(&c, &rows, &rows, kept, at(r), at(r), at(r), at(r), at(r), at(r), at(r), at(r), at(r), at(r), nullptr);
    expect(rc < 0, "conv_bwd with both inputs", rc);
    rc = convseq_scan_bwd(&s, &rows, &rows, nullptr, &rows, nullptr, at(r), at(r), at(r), at(r), at(r), at(r), at(r), at(r),
                          at(r), at(r), nullptr);
    expect(rc < 0, "scan_bwd without a gate", rc);
    rc = convseq_scan_fwd(&s, &rows, &rows, &rows, nullptr, at(r), at(r), at(r), at(r), at(r), kept, at(r), nullptr);
    expect(rc < 0, "scan_fwd without lam", rc);
    rc = convseq_conv_step(&c, at(r), r.next(), nullptr, at(r), at(r), at(r), at(r), pick(), at(r), nullptr);
    expect(rc < 0, "conv_step without w", rc);
    rc = convseq_scan_step(&s, at(r), r.next(), at(r), r.next(), at(r), r.next(), nullptr, at(r), at(r), at(r), pick(), at(r),
                           nullptr);
    expect(rc < 0, "scan_step without lam", rc);
    rc = convseq_pack8(c.b, c.t, c.c, c.dtype, nullptr, kept, nullptr);
    expect(rc < 0, "pack8 without x", rc);
    rc = convseq_unpack8(c.b, c.t, c.c, c.dtype, nullptr, at(r), nullptr);
    expect(rc < 0, "unpack8 without q", rc);
    // empty batches are fine whatever else they hold
    c = {0, r.of(100), 1 + r.of(100), 1 + r.of(8), r.of(2), r.of(3)};
    const convseq_rows none = {nullptr, 0, 0};
    rc = convseq_conv_fwd(&c, &none, (void*)(4096), nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
    expect(rc == 0, "empty conv_fwd", rc);
    rc = convseq_pack8(0, c.t, c.c, c.dtype, &none, kept, nullptr);
    expect(rc == 0, "empty pack8", rc);
  }
}

}  // namespace

int main(int argc, char** argv) {
  const int threads = argc > 1 ? atoi(argv[1]) : 4, rounds = argc > 2 ? atoi(argv[2]) : 1000;
  std::vector<std::thread> all;
  for (int i = 0; i < threads; ++i) all.emplace_back(run, i, rounds);
  for (auto& t : all) t.join();
  printf("%ld inconsistent answers\n", wrong.load());
  return wrong.load() != 0;
}
