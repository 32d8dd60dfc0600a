"""The end of a tree attention call whose wait ran out, without a GPU: copies still in flight have
to land before their shared memory is given up.  The kernel's own routine runs on the host
over barriers that count phases as mbarriers do."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "kv_cache_eviction_trig_b200", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "ring.cuh"

// A place's barrier: `fills` copies were issued into it, `done` of them have landed; a test of
// a parity is true once the phase of that parity is not the current one.
struct Place {
  int fills = 0, done = 0, left = 0;   // left: tests until the copy under way lands
  bool test(unsigned parity) {
    if (done < fills && --left <= 0) ++done;
    return ((unsigned)done & 1u) != parity;
  }
};

int main() {
  srand(1);
  int either = 0;
  for (int places : {1, 2, 4, 5, 8})
    for (int issued = 0; issued < 6 * places + 3; ++issued)
      for (int round = 0; round < 20; ++round) {
        std::vector<Place> ring(places);
        for (int i = 0; i < issued; ++i) ++ring[i % places].fills;
        // a place is filled again only once its last copy has been used: at most one under way
        for (Place &p : ring) {
          p.done = p.fills > 0 && rand() % 2 ? p.fills - 1 : p.fills;
          p.left = 1 + rand() % 50;
        }
        for (const Place &p : ring)   // that some parity tests as complete says nothing
          if (p.done < p.fills) {
            Place q = p;
            q.left = 50;
            either += q.test(0) || q.test(1);
          }
        int awaited = 0;
        tria::drain_ring(issued, places, [&](int s, unsigned parity) {
          ++awaited;
          for (int k = 0; k < 2000 && !ring[s].test(parity); ++k) {
          }
        });
        for (const Place &p : ring)
          if (p.done != p.fills) {
            printf("%d places, %d copies: one in flight\n", places, issued);
            return 1;
          }
        if (awaited != (issued < places ? issued : places)) return 2;
      }
  return either > 0 ? 0 : 3;
}
"""


def test_copies_land_before_shared_memory_is_given_up(tmp_path):
    src, exe = tmp_path / "ring.cc", tmp_path / "ring"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_the_kernel_drains_both_rings():
    """Tiles and queries, by the number of copies issued into each."""
    text = open(os.path.join(CSRC, "tree_attention.cu")).read()
    assert "drain_ring(tiles, NS," in text and "drain_ring(queries, QB," in text
