"""The 4-bit paged cache where its numbers are far from ordinary, and what stands beside one another in a batch."""

import numpy as np
import pytest
import torch

import oracle.attn_oracle as A
import oracle.serving_oracle as S
from gated_deltanet_linear_conv_gb300 import gdn
from helpers import np64
from test_gpu_kv4 import BF, F32, close4, cuts, filled, i32, kv4_reference, new_cache, packed, rand, rope_table, tables

pytestmark = pytest.mark.gpu


def scaled_keys(cache, seed, std):
    """Normal keys of that size in place of the cache's."""
    pages, H, P, half = cache[0].shape
    n, s, m = S.quantise(np64(rand(seed, pages, H, P, 2 * half, dtype=F32)) * std)
    cache[0].copy_(torch.from_numpy(packed(n)))
    cache[2].copy_(torch.from_numpy(np.stack([s, m], -1)))


@pytest.mark.parametrize('D', [64, 128, 256])
@pytest.mark.parametrize('qp,kp', [(113, -114), (117, -118), (121, -122), (126, -127), (-113, 110), (-117, 114), (-121, 118),
                                   (-126, 122), (-131, 124)])
@pytest.mark.parametrize('scale', [None, 1.0])
def test_queries_of_any_size(D, qp, kp, scale):
    """Queries next to either end of float32's range over keys that keep the scores ordinary, large ones beside ordinary
    ones.  (Keys below 2^-100 have no steps: their groups are of one value each.  Queries of 2^-131 have three bits.)"""
    P, H, G, new, lens = 16, 2, 5, [1, 3], [700, 65]
    bt, pages = tables(3, lens, P)
    cache = filled(11, pages, H, P, D)
    scaled_keys(cache, 13, 2.0 ** kp * (1.0 if scale is None else D ** -0.5))
    q = rand(17, sum(new), H * G, D, dtype=F32)
    (q[:, ::3] if qp > 0 else q).mul_(2.0 ** qp)
    q = q.to(BF)
    assert q.isfinite().all()
    y = gdn.paged_kv4_attn_decode(q, *cache, i32(bt.tolist()), i32(lens), cu_seqlens=i32(cuts(new)), scale=scale)
    close4(y, kv4_reference(q, cache, bt, cuts(new), lens, D ** -0.5 if scale is None else scale, None))
    gdn.check_device_error()


@pytest.mark.parametrize('D', [64, 128, 256])
@pytest.mark.parametrize('qp', [100, 117, 121, 124])
@pytest.mark.parametrize('scale', [None, 1.0])
def test_scores_of_large_queries_pick_one_key(D, qp, scale):
    """Keys with steps under such queries: the scores are finite in float32 and lie so far apart that one key takes all."""
    P, H, G, n = 16, 1, 8, 300
    bt, pages = tables(4, [n], P)
    cache = filled(21, pages, H, P, D)
    scaled_keys(cache, 23, 2.0 ** -12)
    q = (rand(27, 1, H * G, D, dtype=F32).sign() * 2.0 ** qp).to(BF)
    y = np64(gdn.paged_kv4_attn_decode(q, *cache, i32(bt.tolist()), i32([n]), scale=scale))
    gdn.check_device_error()
    j = np.arange(n)
    value = [S.values(np.stack([b & 15, b >> 4], -1).reshape(b.shape[:-1] + (D,)), s[..., 0], s[..., 1])
             for b, s in ((c.cpu().numpy(), np64(t)) for c, t in (cache[::2], cache[1::2]))]
    K, V = (x[bt[0][j // P], 0, j % P] for x in value)
    x = np64(q)[0] @ K.T                                     # [heads, tokens]
    assert np.abs(x).max() * (D ** -0.5 if scale is None else scale) * 1.5 < 2.0 ** 128
    top = np.sort(x, -1)
    # float32 sums of D products of size 2^qp (n s + |m|), some 5 or 6 |K|, each rounded by 2^-23 at most: further apart than
    # their errors
    clear = top[:, -1] - top[:, -2] > 2 * (D + 8) * 2.0 ** -23 * 2.0 ** qp * 8 * np.abs(K).sum(-1).max()
    assert clear.sum() >= G // 2
    want = V[x.argmax(-1)]
    # a weight of 1 times a step in f16 (n s of it: V and the group's least value at most), and the output's half step
    near = 2.0 ** -11 * (np.abs(V).max() * 2) + 2.0 ** -8 * np.abs(want)
    assert (np.abs(y[0] - want) <= near)[clear].all()


@pytest.mark.parametrize('D', [64, 128, 256])
@pytest.mark.parametrize('weight', [1.0, 1.5, -2.0])
@pytest.mark.parametrize('spread', [1e-7, 2e-7, 1e-6, 3e-5])
def test_append_bits_of_nearly_constant_rows(D, weight, spread):
    """float32 rows whose groups span a few of their values' last digits, through a norm of equal weights: the stored bits are
    float64's, although float32 is off by whole steps."""
    T, P = 96, 16
    g = torch.Generator().manual_seed(D)
    base = torch.tensor([5.0, -3.0, 1000.0, 0.01, 1.0, 7e4])[torch.arange(T) % 6][:, None, None]
    k = (base * (1 + spread * torch.randn(T, 1, D, generator=g))).cuda()
    w = torch.full((D,), weight, device='cuda')
    bt, pages = tables(3, [T], P)
    at = np.arange(T)
    for rot in (0, 32):                                      # (what is rotated spreads; the groups behind it do not)
        cache, tab = new_cache(pages, 1, P, D), rope_table(T, rot) if rot else None
        gdn.paged_kv4_append(k, k, *cache, i32(bt.tolist()), i32([T]), cos_sin=tab, k_norm_w=w)
        gdn.check_device_error()
        n, s, m = S.quantise(A.norm_rope(np64(k), np64(w), float(np.float32(1e-6)), np64(tab), list(range(T)), False))
        assert np.array_equal(np64(cache[2])[bt[0][at // P], :, at % P], np.stack([s, m], -1).astype(np.float64))
        got = cache[0].cpu().numpy()[bt[0][at // P], :, at % P]
        assert np.array_equal(got, packed(n)), (rot, np.argwhere(got != packed(n))[:4].tolist())


@pytest.mark.parametrize('D,Nq,H', [(64, 6, 3), (128, 32, 8), (256, 16, 2)])
def test_rows_of_inactive_slots(D, Nq, H):
    """Zero rows of inactive slots of any number of rows, alone and among others, long tables and short ones."""
    for seqs, most, P in ((3, 700, 16), (40, 33, 20), (300, 5, 16)):
        rng = np.random.default_rng(seqs)
        for table in (1, 1000):                              # (pages of a short table, of one whose units are cut)
            new = rng.integers(0, most, seqs).tolist()
            lens = [n + int(rng.integers(0, 20)) if n and n < 9 and rng.random() < 0.5 else 0 for n in new]
            new[0], lens[0] = 2, 17
            bt, pages = tables(5, lens, P)
            bt = np.concatenate([bt, np.zeros((seqs, max(0, table // P - bt.shape[1])), np.int64)], 1)
            cache = filled(31, pages, H, P, D)
            T, cu = sum(new), cuts(new)
            q = rand(33, T, Nq, D)
            o = torch.full((T + 3, Nq, D), float('nan'), dtype=BF, device='cuda')
            y = gdn.paged_kv4_attn_decode(q, *cache, i32(bt.tolist()), i32(lens), cu_seqlens=i32(cu), o=o[:T])
            gdn.check_device_error()
            assert o[T:].isnan().all()
            for s, n in enumerate(lens):
                if n == 0:
                    assert (y[cu[s]:cu[s + 1]] == 0).all(), s
            live = [t for s, n in enumerate(lens) if n for t in range(cu[s], cu[s + 1])]
            some = [s for s, n in enumerate(lens) if n][:20]
            ref = kv4_reference(torch.cat([q[cu[s]:cu[s + 1]] for s in some]), cache, bt[some], cuts([new[s] for s in some]),
                                [lens[s] for s in some], D ** -0.5, None)
            close4(torch.cat([y[cu[s]:cu[s + 1]] for s in some]), ref)
            assert y[live].isfinite().all()


def test_a_large_inactive_slot_does_not_hold_the_call():
    """The rest of a step's rows as one inactive slot, 4000 rows of 32 heads of 128 (33 MB): the whole grid clears them.  One
    warp alone writes 256 bytes a step, 128,000 of them: milliseconds.  The limit is a hundred times what a fill takes."""
    D, Nq, H, P, rest = 128, 32, 8, 16, 4000
    lens = [40, 300, 0]
    bt, pages = tables(6, lens, P)
    cache = filled(41, pages, H, P, D)
    q = rand(43, rest + 2, Nq, D)
    args = (q, *cache, i32(bt.tolist()), i32(lens))
    o = torch.empty_like(q)
    run = lambda: gdn.paged_kv4_attn_decode(*args, cu_seqlens=i32([0, 1, 2, rest + 2]), o=o)  # noqa: E731
    times = []
    for _ in range(7):
        run()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        run()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    assert min(times) < 0.6, times
    assert (o[2:] == 0).all() and o[:2].abs().sum() > 0
    gdn.check_device_error()


@pytest.mark.parametrize('D,G', [(64, 3), (128, 8), (256, 8), (64, 16)])
def test_a_sequence_alone_and_in_company(D, G):
    """Cuts and sums go by the batch, so bits may differ with it; the row is right in each."""
    P, H, new = 16, 2, [1, 2, 1, 3]
    lens = [1500, 40, 700, 90]
    bt, pages = tables(8, lens, P)
    cache = filled(51, pages, H, P, D)
    cache[3][bt[2][:3]] *= 2.0 ** 30                         # (a neighbour with other numbers)
    cu = cuts(new)
    q = rand(53, cu[-1], H * G, D)
    y = gdn.paged_kv4_attn_decode(q, *cache, i32(bt.tolist()), i32(lens), cu_seqlens=i32(cu))
    for s in range(4):
        part = q[cu[s]:cu[s + 1]].contiguous()
        ref = kv4_reference(part, cache, bt[s:s + 1], [0, new[s]], lens[s:s + 1], D ** -0.5, None)
        alone = gdn.paged_kv4_attn_decode(part, *cache, i32(bt[s:s + 1].tolist()), i32(lens[s:s + 1]))
        close4(alone, ref, ('alone', s))
        close4(y[cu[s]:cu[s + 1]], ref, ('in company', s))
    gdn.check_device_error()


@pytest.mark.parametrize('D,H', [(64, 5), (128, 2), (256, 1)])
@pytest.mark.parametrize('dtype', [BF, F32])
def test_read_of_keys_or_values_alone(D, H, dtype):
    """One output NULL: the other as with both, and nothing behind either."""
    lens, P = [37, 1, 0, 800], 16
    bt, pages = tables(9, lens, P)
    cache, T, cu = filled(61, pages, H, P, D), sum(lens), i32(cuts(lens))
    table, n = i32(bt.tolist()), i32(lens)
    both = gdn.paged_kv4_read(*cache, table, n, T, cu_seqlens=cu, out_dtype=dtype)
    st, ss = cache[0].stride(), cache[2].stride()
    c = gdn.gdn_paged_cache4(*(t.data_ptr() for t in cache), st[0], st[1], st[2], ss[0], ss[1], ss[2], pages, P, bt.shape[1],
                             table.data_ptr(), n.data_ptr())
    for i in range(2):
        out = torch.full((T + 2, H, D), -7.0, dtype=dtype, device='cuda')
        at = [out.data_ptr() if i == j else None for j in range(2)]
        assert gdn.lib().gdn_paged_kv4_read(gdn.gdn_attn_dims(len(lens), T, H, H, D), cu.data_ptr(), c, *at,
                                            gdn.GDN_BF16 if dtype == BF else gdn.GDN_F32,
                                            torch.cuda.current_stream().cuda_stream) == 0
        gdn.check_device_error()
        assert torch.equal(out[:T], both[i]) and (out[T:] == -7).all()
