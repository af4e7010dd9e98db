"""Inactive slots of many rows in the 16-bit paged attention: a padded step has its unused rows in one."""

import numpy as np
import pytest
import torch

import oracle.attn_oracle as A
from gated_deltanet_linear_conv_gb300 import gdn
from helpers import np64
from test_gpu_paged_attention import BF, F32, Cache, close_attn, cuts, i32, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize('D,Nq,H', [(64, 6, 3), (128, 16, 4), (256, 8, 2)])
@pytest.mark.parametrize('dtype,out_dtype', [(BF, BF), (BF, F32), (F32, F32)])
def test_rows_of_inactive_slots(D, Nq, H, dtype, out_dtype):
    """Zero rows of inactive slots of any number of rows, alone and among others."""
    for seqs, most in ((3, 700), (40, 33), (300, 5)):
        rng = np.random.default_rng(seqs)
        new = rng.integers(0, most, seqs).tolist()
        lens = [n + int(rng.integers(0, 20)) if n and n < 9 and rng.random() < 0.5 else 0 for n in new]
        new[0], lens[0] = 2, 17
        c = Cache([max(1, n) for n in lens], H, 16, D, dtype).fill(lens, 5)
        T, cu = sum(new), cuts(new)
        q = rand(33, T, Nq, D, dtype=dtype)
        o = torch.full((T + 3, Nq, D), float('nan'), dtype=out_dtype, device='cuda')
        y = gdn.paged_attn_decode(q, c.k, c.v, c.block_table, i32(lens), cu_seqlens=i32(cu), out_dtype=out_dtype, o=o[:T])
        gdn.check_device_error()
        assert o[T:].isnan().all()
        for s, n in enumerate(lens):
            if n == 0:
                assert (y[cu[s]:cu[s + 1]] == 0).all(), s
        some = [s for s, n in enumerate(lens) if n][:20]
        part = lambda x: torch.cat([x[cu[s]:cu[s + 1]] for s in some])  # noqa: E731
        ref = A.attention(np64(part(q)), np64(c.k), np64(c.v), c.bt[some], cuts([new[s] for s in some]), [lens[s] for s in some],
                          D ** -0.5, None)
        close_attn(part(y), ref, max(lens), D, dtype, out_dtype)


@pytest.mark.parametrize('dtype', [BF, F32])
def test_a_large_inactive_slot_does_not_hold_the_call(dtype):
    """4000 rows of 32 heads of 128 (33 or 66 MB) cleared by the whole grid.  One warp alone took 12 ms and more; the limit is a
    hundred times what a fill takes."""
    D, Nq, H, rest = 128, 32, 8, 4000
    lens = [40, 300, 0]
    c = Cache([40, 300, 1], H, 16, D, dtype).fill(lens, 5)
    q = rand(43, rest + 2, Nq, D, dtype=dtype)
    o = torch.empty_like(q)
    run = lambda: gdn.paged_attn_decode(q, c.k, c.v, c.block_table, i32(lens), cu_seqlens=i32([0, 1, 2, rest + 2]),  # noqa: E731
                                        out_dtype=dtype, o=o)
    times = []
    for _ in range(7):
        run()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        run()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    assert min(times) < 0.9, times
    assert (o[2:] == 0).all() and o[:2].abs().sum() > 0
    gdn.check_device_error()
