"""Where an expert's blocks begin (csrc/segments.h), for plans as the planner writes them and for ids in any order: the
kernels read sorted_token_ids at what comes out, so it has to stay inside the plan."""
import os
import random
import shutil
import subprocess

import pytest

import mixture_experts_ffn_planner_b200._build as build

PROGRAM = r"""
#include <cstdio>
#include "segments.h"
int main() {  // E, blocks, ids -> the entries that every block sets; then the blocks of every pair "lo hi" that follows
  int E, blocks;
  while (std::scanf("%d %d", &E, &blocks) == 2) {
    int before = -1, here = 0;
    for (int b = 0; b <= blocks; ++b) {
      if (b < blocks && std::scanf("%d", &here) != 1) return 1;
      const moe::SegmentEntries s = moe::segment_entries(b, blocks, E, before, here);
      std::printf("%d %d\n", s.lo, s.hi);
      before = here;
    }
  }
  return 0;
}
"""
BLOCKS = r"""
#include <cstdio>
#include "segments.h"
int main() {
  int lo, hi;
  while (std::scanf("%d %d", &lo, &hi) == 2) std::printf("%d\n", moe::segment_blocks(lo, hi));
  return 0;
}
"""


def _compile(tmp, name, text):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp / f"{name}.cpp", tmp / name
    src.write_text(text)
    subprocess.run([cxx, "-std=c++17", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    return str(exe)


def _run(exe, text):
    return [int(v) for v in subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()]


def _plans():
    rng = random.Random(3)
    for i in range(400):
        E, blocks = rng.randint(1, 12), rng.randint(0, 20)
        ids = [rng.randint(0, E - 1) for _ in range(blocks)]
        if i % 4 == 0:
            ids = sorted(ids)                                  # as the planner writes them
        elif i % 4 == 1:
            ids = [rng.randint(-3, E + 3) for _ in ids]
        elif i % 4 == 2:
            ids = sorted((rng.randint(-1, E) for _ in ids), reverse=True)
        yield i % 4 == 0, E, ids


def test_every_entry_is_set_and_in_range(tmp_path):
    entries, blocks_of = _compile(tmp_path, "entries", PROGRAM), _compile(tmp_path, "blocks", BLOCKS)
    for sound, E, ids in _plans():
        out = _run(entries, " ".join(map(str, [E, len(ids)] + ids)))
        spans = list(zip(out[::2], out[1::2]))
        assert len(spans) == len(ids) + 1
        values = [set() for _ in range(E + 1)]
        for b, (lo, hi) in enumerate(spans):
            for e in range(lo, hi + 1):
                assert 0 <= e <= E, "an entry outside the table is written"
                values[e].add(b)
        assert all(values), f"an entry is never set: {ids}"
        first = [min(v) for v in values]
        pairs = list(zip(first, first[1:]))
        for (lo, hi), n in zip(pairs, _run(blocks_of, "\n".join(f"{a} {b}" for a, b in pairs))):
            assert n >= 0 and (n == 0 or (0 <= lo and lo + n <= len(ids))), (ids, lo, hi, n)
        if sound:
            assert all(len(v) == 1 for v in values)
            assert first == [sum(i < e for i in ids) for e in range(E + 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("K,N", [(64, 96), (512, 768)])  # weight gradients on single CTAs, and on pairs
def test_ids_in_any_order_keep_to_the_plan(K, N):
    """Ids that do not ascend give no gradient that means anything, but every call ends, writes no row behind the
    plan's and leaves the next call right."""
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    E, bm, blocks = 5, 16, 12
    g = torch.Generator(device="cuda").manual_seed(1)
    cap = (blocks + 2) * bm
    ids = torch.arange(cap, dtype=torch.int32, device="cuda")
    total = torch.tensor([blocks * bm], dtype=torch.int32, device="cuda")
    rows = torch.randn((cap, K), generator=g, device="cuda").bfloat16()
    gh = torch.randn((cap, N), generator=g, device="cuda").bfloat16()
    w1 = torch.randn((E, N, K), generator=g, device="cuda").bfloat16()

    def call(experts):
        e = torch.tensor(experts, dtype=torch.int32, device="cuda")
        out = torch.full((cap, K), 3.0, dtype=torch.bfloat16, device="cuda")
        gw = moe.moe_expert_up_backward(gh, rows, w1, ids, e, total, bm, grad_rows=out)[1]
        moe.moe_device_status()
        assert bool((out[blocks * bm:] == 3).all())
        return gw

    sound = sorted(i % E for i in range(blocks)) + [-1, -1]
    want = call(sound)
    for bad in ([4, 3, 2, 1, 0] * 2 + [1, 0], [-1, 0, 3, 0, 9, 2, -7, 4, 4, 1, 0, 0], [4] * 6 + [0] * 6):
        call(bad + [-1, -1])
    assert torch.equal(call(sound), want)
