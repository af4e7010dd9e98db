"""Step metadata and verification where their numbers or inputs are far from ordinary."""

import pytest
import torch

import oracle.serving_oracle as S
from gated_deltanet_linear_conv_gb300 import gdn

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device='cuda')


@pytest.mark.parametrize('new,fits', [([2 ** 30 + 10] * 2, False), ([2 ** 30] * 3, False), ([2 ** 31 - 1, 1], False),
                                      ([2 ** 30 - 1, 2 ** 30], True), ([1, 2 ** 31 - 3, 1], True), ([2 ** 31 - 2, 1], True)])
@pytest.mark.parametrize('where', [0, 600])
def test_plan_sums_next_to_32_bits(new, fits, where):
    """Requests of more tokens than total_tokens = 2^31 - 1 are refused whole, those of as many are not.  (The last sequence alone
    asking for 2^31 - 1 is PLAN_REST.)"""
    N, P, W = where + len(new), 1 << 26, 32
    new = [0] * where + new
    held = [0] * N
    lens, hold, ring, free, table = i32(held), i32(held), i32([0, 128]), torch.arange(128, dtype=torch.int32, device='cuda'), i32([[9] * W] * N)
    out = gdn.PagedPlan(torch.empty(N + 1, dtype=torch.int32, device='cuda'), None, None, *(torch.full((n,), -7, dtype=torch.int32, device='cuda')
                                                                                           for n in (N, N, 2)))
    total = 2 ** 31 - 1
    gdn.paged_plan(i32(new), lens, hold, ring, free, table, P, total, out=out)
    if fits:
        gdn.check_device_error()
        pages = [-(-n // P) for n in new]
        assert out.cu_seqlens.tolist() == [sum(new[:i]) for i in range(N + 1)] and out.kv_lens.tolist() == new
        assert out.pages_held.tolist() == pages and out.free_ring.tolist() == [sum(pages), 128 - sum(pages)]
        assert [p for s, n in enumerate(pages) for p in table[s, :n].tolist()] == list(range(sum(pages)))
    else:
        with pytest.raises(RuntimeError, match='device error 4'):
            gdn.check_device_error()
        assert out.cu_seqlens.tolist() == [0] * (N + 1) and out.kv_lens.tolist() == held and out.pages_held.tolist() == held
        assert out.free_ring.tolist() == [0, 128] and (table == 9).all()


def test_verify_draft_probs_of_no_drafts():
    """A step without drafts: the same as with none given; with drafts the call is refused."""
    N, V = 5, 300
    g = torch.Generator().manual_seed(1)
    p, u = torch.softmax(torch.randn(2 * N, V, generator=g), -1).cuda(), torch.rand(2 * N, generator=g).cuda()
    tok, none = i32([3] * (2 * N)), torch.empty(N, 0, V, device='cuda')
    acc, out, _ = gdn.draft_verify(p[:N], tok[:N], u[:N], none, num_seqs=N)
    assert acc.tolist() == [0] * N and torch.equal(out, gdn.draft_verify(p[:N], tok[:N], u[:N], num_seqs=N)[1])
    gdn.draft_verify(p[:1], tok[:1], u[:1], none, cu_seqlens=i32([0, 0, 1, 1, 1, 1]))
    gdn.draft_verify(p[:0], tok[:0], u[:0], none, cu_seqlens=i32([0] * (N + 1)))
    for T, cu in ((2 * N, None), (N, i32([0, 2, 3, 4, 5, 5])), (N, i32([0, 1, 2, 3, 4, 5]))):
        with pytest.raises(ValueError, match='no drafts'):
            gdn.draft_verify(p[:T], tok[:T], u[:T], none, cu_seqlens=cu, num_seqs=N)
    gdn.check_device_error()


@pytest.mark.parametrize('bad', [-1, 12, 2 ** 31 - 1])
@pytest.mark.parametrize('seqs', [3, 700])
def test_plan_page_out_of_range_given_back(bad, seqs):
    """An ended sequence's page that is none of the cache's is flagged when it goes back, not when it is given out."""
    new, held = [-1] + [0] * (seqs - 1), [2] + [0] * (seqs - 1)
    table = torch.zeros(seqs, 3, dtype=torch.int32, device='cuda')
    table[0, :2] = i32([3, bad])
    for row, flagged in ((0, True), (seqs - 1, False)):      # of a sequence that has ended, or lies idle
        free = torch.full((12,), -9, dtype=torch.int32, device='cuda')
        t, n, h = table.clone(), list(new), list(held)
        if row:
            t[row], t[0], n[row], h[row] = table[0], i32([3, 4, 0]), 0, 2
        out = gdn.paged_plan(i32(n), i32([5 if x else 0 for x in h]), i32(h), i32([11, 0]), free, t, 4, 0)
        if flagged:
            with pytest.raises(RuntimeError, match='device error 3'):
                gdn.check_device_error()
        else:
            gdn.check_device_error()
        assert out.free_ring.tolist() == [11, 2] and [int(free[11]), int(free[0])] == [3, bad if flagged else 4]
        assert out.pages_held.tolist()[0] == 0 and out.kv_lens.tolist()[0] == 0


def test_a_step_of_prompts_and_drafts():
    """Prompts beside sequences with drafts: the plan's bounds count every token, the verification's the rows with
    probabilities, one of a prompt.  Lengths and the next step against the oracles."""
    N, P, V, W = 5, 8, 200, 12
    gen = torch.Generator().manual_seed(3)
    pages = N * W
    st = dict(lens=[0] * N, held=[0] * N, ring=[0, pages], free=torch.randperm(pages, generator=gen).tolist(), table=[[0] * W for _ in range(N)])
    dev = {k: i32(v) for k, v in st.items()}
    for new, prompt in (([20, 0, 9, 0, 1], {0, 2, 4}), ([4, 17, 4, 0, 3], {1}), ([4, 3, -1, 30, 1], {3}), ([2, 4, 5, 4, -1], {2})):
        T = sum(max(n, 0) for n in new)
        plan = gdn.paged_plan(i32(new), dev['lens'], dev['held'], dev['ring'], dev['free'], dev['table'], P, T)
        ref = S.plan(new, page_size=P, total=T, **st)
        assert plan.cu_seqlens.tolist() == ref['cu'] and plan.kv_lens.tolist() == ref['lens']
        last = [list(range(a, b))[-1 if s in prompt else 0:] for s, (a, b) in enumerate(zip(ref['cu'], ref['cu'][1:]))]
        rows = [t for r in last for t in r]
        cu = [sum(map(len, last[:s])) for s in range(N + 1)]
        p = torch.softmax(torch.randn(T, V, generator=gen) * 2, -1)[rows]
        tok, u = torch.randint(V, (T,), generator=gen, dtype=torch.int32)[rows], torch.rand(T, generator=gen)[rows]
        acc, out, lens = gdn.draft_verify(p.cuda(), tok.cuda(), u.cuda(), cu_seqlens=i32(cu), kv_lens=plan.kv_lens)
        racc, rout, rlens = S.verify(p.double().numpy(), tok.tolist(), u.double().tolist(), None, cu, ref['lens'])
        assert (acc.tolist(), out.tolist(), lens.tolist()) == (racc, rout, rlens)
        for s in prompt:
            assert acc[s] == 0 and out[cu[s]] >= 0 and rlens[s] == ref['lens'][s]          # all of a prompt stays
        st = dict(lens=rlens, **{x: ref[x] for x in ('held', 'ring', 'free', 'table')})
        dev.update(lens=lens, held=plan.pages_held, ring=plan.free_ring)
        assert dev['table'].tolist() == ref['table']
    gdn.check_device_error()
