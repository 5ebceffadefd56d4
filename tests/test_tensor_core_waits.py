"""The matrix product's barrier waits, read from its source: what cannot be shown on a GPU without
a wait that runs out in the middle of a kernel."""
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_epilogue_gb300", "csrc")


def code(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_waits_are_a_whole_warp_s():
    """A bounded wait ends by the clock, lane by lane: what follows it is for whole warps (aligned loads of tensor memory,
    elections, barriers of the cluster), so all lanes have to take the same way out."""
    src = code("matmul.cu")
    assert not re.findall(r"\bmbar_(?:try_)?wait\w*\s*\(", src)
    assert len(re.findall(r"\bwarp_wait\(", src)) >= 8
    wait = re.search(r"bool warp_wait\([^)]*\)\s*\{(.*?)\}", code("umma.cuh"), re.S).group(1)
    assert "__all_sync(0xffffffffu, mbar_wait(" in wait


PROGRAM = r"""
#include <cstdio>
#include "ring_tail.h"
struct Ring { int st = 0; unsigned phase = 0; int n; explicit Ring(int s) : n(s) {}
              void next() { if (++st == n) { st = 0; phase ^= 1u; } } };
int main() {
  for (int n = 1; n <= 8; ++n)
    for (int items = 0; items <= 5 * n + 3; ++items) {
      Ring ring(n);
      for (int i = 0; i < items; ++i) ring.next();
      const int uses = items < n ? items : n;
      int i = items - uses, seen = 0;
      const bool all = ep::dev::last_uses(ring, uses, [&](int st, uint32_t parity) {
        const bool good = st == i % n && parity == unsigned(i / n & 1);  // item i: stage i % n, use i / n
        ++i;
        ++seen;
        return good;
      });
      if (!all || seen != uses) return 1;
      // a refusal ends it
      seen = 0;
      if (ep::dev::last_uses(ring, uses, [&](int, uint32_t) { return ++seen < 2; }) != (uses < 2)) return 2;
      if (seen != (uses < 2 ? uses : 2)) return 3;
    }
  std::puts("ok");
}
"""


def test_the_last_uses_of_a_ring(tmp_path):
    (tmp_path / "main.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "main")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(tmp_path / "main.cpp"), "-o", exe], check=True,
                   timeout=120)
    assert subprocess.run([exe], capture_output=True, text=True, timeout=60).stdout.strip() == "ok"


def body(src, kernel):
    at = src.index(f"{kernel}(const __grid_constant__")
    return src[at:src.index("\n}\n", at)]


def test_every_barrier_s_last_arrivals_are_waited_for():
    """What the tensor cores send to a barrier when they are done lands before the CTA that holds it leaves: each
    barrier of a commit has a wait for its last uses in every CTA that the commit arrives in."""
    src = code("matmul.cu")
    pair, split = body(src, "k_mm_pair"), body(src, "k_mm_split")
    tail = r"last_uses\(ring, issued, \[&\]\(int st, uint32_t parity\) \{ return warp_wait\(%s \+ st, parity\)(?: \|\| true)?; \}\);"
    assert set(re.findall(r"mma_commit<true>\((\w+)", pair)) == {"empty", "ready", "drained"}
    assert set(re.findall(r"mma_commit<false>\(&?(\w+)", split)) == {"sempty", "empty", "done"}
    for kernel, bars in ((pair, ("full", "empty")), (split, ("full", "empty", "sempty"))):
        for bar in bars:
            assert len(re.findall(tail % bar, kernel)) == 1, bar
    # both CTAs of a pair: no condition on the rank in front of it (the loads arrive in the first alone)
    assert re.search(r"\n    last_uses\([^\n]*empty", pair) and re.search(r"if \(rank == 0\) last_uses\([^\n]*full", pair)
    # (an accumulator's `ready` is waited for by the warps that write it, in both; `drained` and `done` by who sends them)
    assert "warp_wait(ready + acc" in pair and "mma_commit<true>(drained, 1)" in pair and "warp_wait(&done, 0)" in split
