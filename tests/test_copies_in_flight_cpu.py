"""The producers' record of copies in flight (csrc/copies_in_flight.cuh), compiled for
the host and run against a model of the mbarriers: after a wait that ran out at any
moment, drain() returns only when every issued copy has landed, and gives up where one
never does.  The model's parity wait succeeds while the phase of that parity is the
last completed one, so that asking for either parity waits for nothing.
"""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "recurrent_memory_transformer_diag_b200", "csrc")

HARNESS = r"""
#include "copies_in_flight.cuh"
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

struct Bar {
  int phase = 0;       // number of completed phases
  int lands_at = -1;   // time at which the copy in flight lands
  bool done(unsigned parity) const { return ((phase & 1) != 0) != (parity != 0); }   // phase - 1 has this parity
};

int main() {
  std::mt19937 rng(7);
  long waited = 0, either = 0, cases = 0;
  for (int trial = 0; trial < 20000; ++trial) {
    const int stages = 1 + rng() % 12, total = rng() % 60, stop_at = rng() % 120;
    const bool lost = trial % 50 == 0;    // the last copy never lands
    std::vector<Bar> bar(stages);
    armt::CopiesInFlight copies;
    int now = 0, sent = 0, used = 0, last = 0;
    auto tick = [&] {
      ++now;
      for (auto& b : bar)
        if (b.lands_at >= 0 && b.lands_at <= now) { b.lands_at = -1; ++b.phase; }
    };
    for (; now < stop_at; tick()) {       // the producer and the consumer until somebody gives up
      if (sent < total && sent - used < stages && rng() % 3) {
        const int s = sent % stages, round = sent / stages;
        bar[s].lands_at = now + 1 + rng() % 9;
        copies.issued(s, round & 1);
        last = s;
        ++sent;
      }
      if (used < sent && bar[used % stages].done(used / stages & 1) && rng() % 3) ++used;
    }
    if (lost && sent && bar[last].lands_at >= 0) bar[last].lands_at = 1 << 30;
    bool flying = false, forever = false;
    for (auto& b : bar) { flying |= b.lands_at >= 0; forever |= b.lands_at == 1 << 30; }
    if (flying) {
      ++cases;
      for (int s = 0; s < stages; ++s) either += bar[s].lands_at >= 0 && (bar[s].done(0) || bar[s].done(1));
    }
    const int t0 = now;
    const bool ok = copies.drain([&](int s, uint32_t par) { return bar[s].done(par); },
                                 [&] { tick(); return now - t0 > 100; });
    waited += now - t0;
    for (auto& b : bar)
      if (b.lands_at >= 0 && b.lands_at != 1 << 30) { printf("a copy in flight after drain\n"); return 1; }
    if (ok == forever) { printf("drain says %d\n", ok); return 1; }
  }
  printf("%ld %ld %ld\n", cases, either, waited);
  return 0;
}
"""


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    d = tmp_path_factory.mktemp("copies")
    src, exe = d / "model.cpp", d / "model"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)


def test_drain_waits_for_every_copy(model):
    assert model.returncode == 0, model.stdout
    cases, either, waited = map(int, model.stdout.split())
    assert cases > 5000 and waited > cases    # copies were in flight, and waited for
    assert either >= cases                    # what asking for either parity would have let pass


@pytest.mark.parametrize("name,producers", [("tc_gemm.cu", 2), ("attention_tc.cu", 1), ("token_loss.cu", 2)])
def test_producers_keep_that_record(name, producers):
    text = open(os.path.join(CSRC, name)).read()
    assert text.count("CopiesInFlight copies;") == text.count("copies.drain(") == producers
    assert text.count("copies.issued(") >= producers
    # a barrier is never asked for either parity
    assert not re.search(r"try_wait\w*(<\w+>)?\([^;\n]*, 0\) (&&|\|\|) !?mbar_try_wait\w*\([^;\n]*, 1\)", text)
