"""Corners of the operators of include/ar_ops.h on the GPU: values, streams, captures and rows at the edge of what
each is specified for, against the same 64-bit implementations as test_gpu_ops.py."""
import math

import numpy as np
import pytest
import torch

from tests import ops_helpers as H
from tests.test_gpu_ops import _attend_case, _check_attend, _gen, _i32, _tda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 2)])
def test_attend_many_segments_to_a_warp(window, sinks):
    """8192 short requests: every warp walks through several segments, whole ones and parts.  The requests repeat 64
    different ones (page ids may), so that the plain implementation need not run 8192 times."""
    tda = _tda()
    kinds, B, D = 64, 8192, 64
    g = np.random.RandomState(3)
    lens = [int(x) for x in g.randint(1, 150, kinds)]
    q, pool, K, V, table, cu = _attend_case(47, kinds, lens, [1] * kinds, 2, 4, D, 16, "bf16")
    want, wl, mag, big, top = H.attend(q, K, V, table, lens, cu, window, sinks, D ** -0.5)
    bo, bl = H.attend_bounds(want, wl, mag, big, top, D ** -0.5, q.dtype, max(lens))
    pick = torch.from_numpy(g.randint(0, kinds, B))
    out, lse = tda.kv4_attend(q[pick].cuda(), pool.cuda(), _i32(table)[pick.cuda()], _i32(lens)[pick.cuda()], window=window,
                              sinks=sinks, return_lse=True)
    assert ((out.cpu().double() - want[pick]).abs() <= bo[pick]).all()
    assert ((lse.cpu().double() - wl[pick]).abs() <= bl[pick]).all()
