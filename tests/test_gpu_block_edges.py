"""GPU tests of the block norms, 8-bit checkpoints, the weight gradient taken
from one and the gated unit where they can go wrong: kernels that follow one
another closely, gates far from zero, guard bytes around every output.

Tolerances are those of test_gpu_block.py unless a test derives its own.
"""
import numpy as np
import pytest
import torch

import deterministic_attention_gb300 as da
from helpers import to_np
from oracle import block as ob
from test_gpu_block import BF, F32, U, _acts, _gen, _within

# ------------------------------------------------------------ weight gradient


@pytest.mark.gpu
def test_wgrad_blocks_leave_nothing_behind_for_the_next_kernel():
    """Launches that follow one another closely on two streams, so that blocks
    take over shared memory which a pair has just left: a barrier that such a
    pair's products still reached would be counted wrong.  Few steps (fewer
    than the rings are deep, and a few more), odd pairs' columns included."""
    g = _gen(61)
    q = torch.randn((1, 512, 4, 64), generator=g).to(BF).cuda()
    a = torch.randn((512, 256), generator=g).to(BF).cuda()
    calls = []
    for rows, d, n in ((1, 32, 8), (64, 512, 512), (200, 2432, 1032), (321, 96, 264), (449, 768, 1280)):
        c = da.act8_pack(_acts(g, rows, d).cuda())
        dy = torch.randn((rows, n), generator=g).to(BF).cuda()
        calls.append(lambda c=c, dy=dy: da.act8_wgrad(c, dy))
    calls.append(lambda: da.attn_fwd(q, q, q)[0])
    calls.append(lambda: da.layer_gemm(a, a[:256].contiguous(), out_fp32=True))
    refs = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for k in range(40):
        outs = []
        for st in streams:
            with torch.cuda.stream(st):
                outs += [f() for f in calls]
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            assert torch.equal(o, refs[i % len(calls)]), (k, i)
    da.check_status()
