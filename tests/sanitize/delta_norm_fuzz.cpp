// delta_norm_fuzz.cpp -- drives the host side of include/convdelta.h and
// include/convnorm.h under sanitizers: random (valid and invalid) descriptors, views
// and buffers through every entry point from several threads.  No call launches:
// each either has something that validation refuses, or describes an empty batch.
//
//   delta_norm_fuzz THREADS ROUNDS
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <atomic>
#include <thread>
#include <vector>

#include "../../include/convdelta.h"
#include "../../include/convnorm.h"

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

void expect(bool ok, const char* what, int64_t rc) {
  if (!ok) {
    ++wrong;
    fprintf(stderr, "%s: %lld\n", what, (long long)rc);
  }
}

// Addresses far apart that nothing reads: validation looks at their values only.
void* at(Rng& r) { return (void*)(((uintptr_t)r.of(64) + 1) << 32); }

void run(int id, int rounds) {
  Rng r{(uint64_t)id * 7919 + 1};
  static const int32_t odd[] = {-2147483647, -1, 0, 1, 2, 15, 16, 17, 64, 128, 1000, 65537, 1 << 22, 1 << 26, 2147483647};
  for (int n = 0; n < rounds; ++n) {
    const auto pick = [&] { return odd[r.of(15)]; };
    const auto some = [&] { return 1 + r.of(20); };
    const auto stride = [&] { return ((int64_t)r.next() << (r.of(3) * 14)) - (r.of(50) == 0); };
    // half of them are sensible but for one extent
    convdelta_desc d = {pick(), pick(), pick(), pick(), pick(), pick(), r.of(5) - 1, r.of(9) ? 1.f : 1e39f};
    if (r.of(2)) {
      d = {some(), some() * 40, some(), 0, 1 + r.of(130), some() * 16, r.of(3), 0.5f};
      d.hv = d.hk * some();
      int32_t* field = &d.b + r.of(6);
      *field = pick();
    }
    const int64_t fw = convdelta_fwd_workspace(&d), bw = convdelta_bwd_workspace(&d);
    expect((fw < 0) == (bw < 0) && fw >= -7, "delta workspace", fw);
    if (fw >= 0) expect(d.hv % d.hk == 0 && d.dk <= CONVDELTA_MAX_DK && d.b >= 0 && d.t >= 0, "delta desc", fw);
    const convdelta_heads h = {at(r), stride(), stride(), stride()};
    int rc;
    if (d.b > 0 && d.t > 0) {
      rc = convdelta_fwd(&d, &h, &h, &h, at(r), nullptr, at(r), at(r), at(r), at(r), at(r), at(r), at(r), nullptr);
      expect(rc < 0, "delta_fwd without beta", rc);
      rc = convdelta_fwd(&d, &h, nullptr, &h, at(r), at(r), at(r), at(r), at(r), at(r), at(r), at(r), at(r), nullptr);
      expect(rc < 0, "delta_fwd without k", rc);
      rc = convdelta_bwd(&d, &h, &h, &h, &h, at(r), at(r), nullptr, at(r), at(r), at(r), at(r), at(r), at(r), at(r), at(r),
                         at(r), at(r), nullptr);
      expect(rc < 0, "delta_bwd without states", rc);
      void* same = at(r);
      rc = convdelta_step(&d, &h, &h, &h, at(r), at(r), same, same, at(r), some(), same, nullptr);
      expect(rc < 0, "delta_step without room", rc);
    }
    convnorm_desc m = {pick(), pick(), pick(), pick(), r.of(4) - 1, r.of(5) - 1, r.of(5) - 1, r.of(9) ? 1e-5f : -1.f};
    if (r.of(2)) {
      m = {some(), some() * 100, 0, some(), r.of(2), r.of(3), 0, 1e-5f};
      m.c = m.groups * some();
      int32_t* field = &m.n + r.of(3);
      *field = pick();
    }
    const int64_t nf = convnorm_group_fwd_workspace(&m), nb = convnorm_group_bwd_workspace(&m);
    expect(nf >= -7 && nb >= -7, "norm workspace", nf);
    if (nf >= 0) expect(m.c % m.groups == 0 && m.n >= 0 && m.p >= 0, "norm desc", nf);
    const convseq_rows rows = {at(r), stride(), stride()};
    if (m.n > 0) {
      rc = convnorm_group_fwd(&m, &rows, at(r), at(r), at(r), nullptr, at(r), at(r), nullptr);
      expect(rc < 0, "norm_fwd without a mean", rc);
      rc = convnorm_group_bwd(&m, &rows, &rows, at(r), at(r), at(r), nullptr, at(r), at(r), at(r), at(r), nullptr);
      expect(rc < 0, "norm_bwd without rstd", rc);
    }
    // empty batches are fine whatever else they hold
    d = {0, r.of(100), 1 + r.of(4), 0, 1 + r.of(128), 1 + r.of(100), r.of(3), 1.f};
    d.hv = d.hk * (1 + r.of(3));
    const convdelta_heads none = {nullptr, 0, 0, 0};
    rc = convdelta_fwd(&d, &none, &none, &none, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                       nullptr);
    expect(rc == 0, "empty delta_fwd", rc);
    rc = convdelta_step(&d, &none, &none, &none, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr, nullptr);
    expect(rc == 0, "empty delta_step", rc);
    m = {0, r.of(100), 0, 1 + r.of(9), r.of(2), r.of(3), 0, 0.f};
    m.c = m.groups * (1 + r.of(30));
    const convseq_rows nothing = {nullptr, 0, 0};
    rc = convnorm_group_fwd(&m, &nothing, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
    expect(rc == 0, "empty norm_fwd", rc);
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
