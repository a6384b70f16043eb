"""The launch plan of the paged attention as the library computes it (compiled
from its header), and the tiles that each CTA of a call takes."""
import ctypes as C
import functools
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "kernels.h"
extern "C" void plan(int heads_q, int heads_kv, int dim, int *out) {
    const nvfp4::PagedPlan n = nvfp4::paged_plan(heads_q, heads_kv, dim);
    out[0] = n.parts_shift, out[1] = n.ranges, out[2] = n.stages, out[3] = n.blocks;
}
"""
#: tiles that taking up a sequence counts in the schedule
PART_TILES = 3


@functools.cache
def _lib():
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-fPIC", "-shared", "-I", os.path.join(ROOT, "nvfp4_block_scaled_22_b200", "csrc"),
                        "-I", "/usr/local/cuda/include", src, "-o", so], check=True)
        return C.CDLL(so)


def plan(heads_q, heads_kv, dim):
    """(tokens of a tile, ranges, stages, CTAs over the heads)."""
    out = (C.c_int * 4)()
    _lib().plan(heads_q, heads_kv, dim, out)
    return 16 << out[0], out[1], out[2], out[3]


def tiles_of_ranges(lens, heads_q, heads_kv, dim):
    """The tiles of each range, as (sequence, tile) in the order they are taken."""
    tokens, ranges, _, _ = plan(heads_q, heads_kv, dim)
    places = []
    for b, n in enumerate(lens):
        places += [None] * PART_TILES + [(b, t) for t in range(max(1, -(-n // tokens)))]
    n = min(len(places), ranges)
    length, longer = divmod(len(places), n)
    cuts = [x * length + min(x, longer) for x in range(n + 1)]
    return [[p for p in places[a:z] if p] for a, z in zip(cuts, cuts[1:])]
