"""The choice of kernel of paged attention, compiled from its header for the host."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sequence_decode_step_gb300", "csrc")
MAIN = """
#include <cstdio>
#include "paged_plan.h"
int main() {
  int kv, act, nkv, gq, n, seqs, most;
  long long keys;
  while (std::scanf("%d %d %d %d %d %d %d %lld", &kv, &act, &nkv, &gq, &n, &seqs, &most, &keys) == 8) {
    const qw::PagedPlan p = qw::plan_paged_pass(kv, act, nkv, gq, n, seqs, most, keys, 152);
    std::printf("%d %d %d %d\\n", p.tc, p.kt, p.rows, p.grid);
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", str(d / "plan"), str(d / "main.cpp")],
                   check=True)

    def ask(kv, act, nkv, gq, seqs, new, keys, n=None):
        n = seqs * new if n is None else n
        line = f"{kv == 'bf16':d} {act == 'bf16':d} {nkv} {gq} {n} {seqs} {new} {keys}\n"
        out = subprocess.run([str(d / "plan")], input=line, capture_output=True, text=True, check=True).stdout
        tc, kt, rows, grid = map(int, out.split())
        return bool(tc), kt, rows, grid
    return ask


@pytest.mark.parametrize("act,kv,seqs,new,keys", [
    # kernels whose times differ by 2 and more: 158 us against 1 421, 49 against 204, 62 against 166,
    # 150 against 386, 237 against 771, 125 against 492, 47 against 123
    ("bf16", "bf16", 160, 16, 4096), ("bf16", "bf16", 32, 16, 4096), ("bf16", "bf16", 160, 8, 1024),
    ("bf16", "bf16", 160, 4, 4096), ("f32", "bf16", 160, 8, 4096), ("f32", "f32", 160, 16, 1024),
    ("f32", "f32", 32, 16, 1024)])
def test_the_whole_batch_counts(plan, act, kv, seqs, new, keys):
    assert plan(kv, act, 2, 8, seqs, new, keys)[0]


def test_few_rows_and_short_chunks_stay_on_the_decode_kernels(plan):
    for kv in ("bf16", "f32"):
        for seqs in (1, 32, 256):
            assert not plan(kv, "f32", 2, 8, seqs, 1, 8192)[0]
            assert not plan(kv, "f32", 8, 2, seqs, 8, 8192)[0]
    # one sequence alone: 15.0 us against 18.5, 18.4 against 20.6
    assert not plan("bf16", "bf16", 2, 8, 1, 16, 256)[0]
    assert not plan("bf16", "f32", 2, 8, 1, 3, 4096)[0]


def test_a_wrong_hint_is_a_plan_too(plan):
    # more new tokens than there are, and fewer
    assert plan("bf16", "bf16", 2, 8, 4, 1 << 30, 4096, n=64) == plan("bf16", "bf16", 2, 8, 1, 64, 4096)
    assert plan("f32", "f32", 2, 8, 1, 1, 4096, n=500)[1:] == (32, 8, 304)
    assert plan("f32", "f32", 2, 2, 300, 1, 1 << 30, n=300)[1:] == (32, 2, 456)
    assert plan("bf16", "bf16", 8, 8, 1 << 20, (1 << 31) - 1, (1 << 31) - 600, n=1 << 25)[0]
