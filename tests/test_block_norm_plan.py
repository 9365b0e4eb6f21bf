"""The launch that block_norm_plan.py describes is the library's.  No GPU needed."""
import ctypes
import random

import compressed_mixture_experts_amd as bm
from compressed_mixture_experts_amd import blocks
from block_norm_plan import backward_plan
from test_gpu_block_norm_sums import SHAPES


def test_workgroups_are_the_library_s():
    """The workspace has four rows of fp32 for every workgroup."""
    r = random.Random(3)
    sizes = [(r.choice([r.randint(1, 300), r.randint(1, 5000), r.randint(1, 1 << 24)]), r.choice([r.randint(1, 300), r.randint(1, 16384)]))
             for _ in range(20000)]
    for rows, width in sizes + SHAPES:
        n, size = blocks._BlockNorm(rows=rows, width=width), ctypes.c_size_t(0)
        assert bm.lib().bmoe_block_norm_backward_workspace(ctypes.byref(n), ctypes.byref(size)) == 0
        assert size.value == backward_plan(rows, width)[0] * 16 * width, (rows, width)


def test_tested_sizes_loop_in_every_form():
    """Sizes for which workgroups take rows more than once, with a last time that has not all
    of them: in every number of threads a row."""
    def form(width):
        return 0 if width < 8 else sum(width > w for w in (128, 256, 512, 1024, 2048, 4096, 8192)) + 1

    loops = {form(w) for r, w in SHAPES if backward_plan(r, w)[2] > 1}
    ragged = {form(w) for r, w in SHAPES if (b := backward_plan(r, w)) and b[2] > 1 and r % (b[0] * b[1])}
    assert loops == ragged == set(range(9))
