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


# A CTA pair: the copies of both are counted, in bytes, on the even CTA's barriers, which
# the even CTA arms for both; the CTAs stop at different stages.
PAIR = r"""
#include "copies_in_flight.cuh"
#include <cstdio>
#include <random>
#include <vector>

struct Bar {
  int phase = 0, arrived = 0, tx = 0;
  bool twice = false;   // armed again before the phase was complete
  void check() { if (arrived && tx == 0) { ++phase; arrived = 0; } }
  void expect(int bytes) { twice |= arrived != 0; tx += bytes; arrived = 1; check(); }
  void land(int bytes) { tx -= bytes; check(); }
  bool done(unsigned parity) const { return ((phase & 1) != 0) != (parity != 0); }
};
struct Copy { int cta, stage, bytes, at; };

int main() {
  std::mt19937 rng(11);
  long odd_alone = 0, even_alone = 0, armed_late = 0;
  for (int trial = 0; trial < 20000; ++trial) {
    const int stages = 1 + rng() % 7, total = rng() % 40;
    std::vector<Bar> bar(stages);
    std::vector<Copy> flying;
    armt::CopiesInFlight mine[2];
    std::vector<int> bytes(stages);
    int now = 0, sent[2] = {0, 0}, used = 0;
    const int stop[2] = {(int)(rng() % 100), (int)(rng() % 100)};
    auto tick = [&] {
      ++now;
      for (size_t i = 0; i < flying.size();) {
        if (flying[i].at <= now) {
          bar[flying[i].stage].land(flying[i].bytes);
          flying.erase(flying.begin() + i);
        } else {
          ++i;
        }
      }
    };
    for (; now < 100; tick()) {
      for (int c = 0; c < 2; ++c) {
        if (now >= stop[c] || sent[c] >= total || sent[c] - used >= stages || rng() % 3 == 0) continue;
        const int s = sent[c] % stages, size = 3 + sent[c] * 7 % 2;   // of three or four boxes
        if (c == 0) bar[s].expect(2 * size);
        else bytes[s] = size;
        flying.push_back({c, s, size, now + 1 + (int)(rng() % 9)});
        mine[c].issued(s, sent[c] / stages & 1);
        ++sent[c];
      }
      if (used < sent[0] && used < sent[1] && bar[used % stages].done(used / stages & 1)) ++used;
    }
    odd_alone += sent[1] > sent[0];
    even_alone += sent[0] > sent[1];
    auto landed = [&](int s, uint32_t par) { return bar[s].done(par); };
    int t0 = now;
    const bool all = mine[0].drain(landed, [&] { tick(); return now - t0 > 50; });
    if (all != (sent[1] >= sent[0])) { printf("even drain %d\n", all); return 1; }
    if (mine[0].word() != mine[1].word()) {
      const auto rest = armt::CopiesInFlight::of(mine[1].word()).beyond(armt::CopiesInFlight::of(mine[0].word()));
      for (int s = 0; s < stages; ++s)
        if ((rest.stages >> s & 1) && !landed(s, rest.parity >> s & 1)) { bar[s].expect(bytes[s]); ++armed_late; }
      t0 = now;
      if (!rest.drain(landed, [&] { tick(); return now - t0 > 50; })) { printf("rest does not land\n"); return 1; }
    }
    for (auto& b : bar)
      if (b.twice) { printf("armed twice\\n"); return 1; }
    if (!flying.empty()) { printf("%zu copies in flight\n", flying.size()); return 1; }
  }
  printf("%ld %ld %ld\n", odd_alone, even_alone, armed_late);
  return 0;
}
"""


def run(tmp_path_factory, text):
    d = tmp_path_factory.mktemp("copies")
    src, exe = d / "model.cpp", d / "model"
    src.write_text(text)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    return run(tmp_path_factory, HARNESS)


def test_pair_waits_for_copies_of_stages_that_only_the_odd_cta_used(tmp_path_factory):
    r = run(tmp_path_factory, PAIR)
    assert r.returncode == 0, r.stdout
    odd_alone, even_alone, armed_late = map(int, r.stdout.split())
    assert odd_alone > 1000 and even_alone > 1000 and armed_late > 1000


@pytest.mark.parametrize("name", ["tc_gemm.cu", "token_loss.cu"])
def test_pair_kernels_exchange_the_record(name):
    text = open(os.path.join(CSRC, name)).read()
    assert text.count("copies.word()") == 2 and text.count("rest.drain(") == 1
    assert text.index("copies.word()") < text.index("copies.drain(", text.index("copies.word()")) < text.index("rest.drain(")


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
