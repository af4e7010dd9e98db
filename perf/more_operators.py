"""Measured cases of the operators around a 4-bit paged cache and draft + verify decoding.

Five operators, as a serving loop uses them: "plan" (block tables, lengths and slot maps of the next step from the
requests' lengths), "append" (norm, rotation, keys and values into the cache in 4 bits; read back, since what 4 bits
hold is compared as values), "read" (cached tokens as dense keys and values), "attn" (attention of the new tokens
over the cache) and "verify" (which drafted tokens stay, and the token behind them).  ``own`` is set from outside:
false computes the plain form, true calls the library.  Sizes: 256-sequence decode, 16 sequences of 512..8192 tokens
and a 131072-token context are the workloads of inputs.py; head counts, head widths and vocabularies are generic.

The 4-bit cache: k and v [pages, Nkv, page, D/2] uint8 (element 2i in the low half of byte i), scales [pages, Nkv,
page, D/64, 2] bf16: a group of 64 elements with step s and least value m holds n = 0..15 for n s + m.  q [T, Nq, D];
block_table [N, pages per sequence] int32, kv_lens [N] int32 (cached tokens including the call's own).
"""

import bisect
import itertools
import math
import random

import torch

own = False

GROUP = 64


# ------------------------------------------------------------------------------- the cases

def _named(name, c):
    return dict(c, name=name) if name else c


def _plan(name, seqs, lo, hi, new, page, gone, idle, len_seed):
    return _named(name, dict(op='plan', seqs=seqs, lo=lo, hi=hi, new=new, page=page, gone=gone, idle=idle,
                             len_seed=len_seed))


def _verify(name, seqs, lo, hi, vocab, draft, dtype, len_seed):
    return _named(name, dict(op='verify', seqs=seqs, lo=lo, hi=hi, vocab=vocab, draft=draft, dtype=dtype,
                             len_seed=len_seed))


def _append(name, seqs, lo, hi, new, nq, nkv, d, rot, inter, norm, page, dtype, len_seed):
    return _named(name, dict(op='append', seqs=seqs, lo=lo, hi=hi, new=new, nq=nq, nkv=nkv, d=d, rot=rot, inter=inter,
                             norm=norm, page=page, dtype=dtype, len_seed=len_seed))


def _read(name, seqs, lo, hi, nkv, d, page, dtype, len_seed):
    return _named(name, dict(op='read', seqs=seqs, lo=lo, hi=hi, new=0, nkv=nkv, d=d, page=page, dtype=dtype,
                             len_seed=len_seed))


def _attn(name, seqs, lo, hi, new, nq, nkv, d, page, gate, len_seed):
    return _named(name, dict(op='attn', seqs=seqs, lo=lo, hi=hi, new=new, nq=nq, nkv=nkv, d=d, page=page, gate=gate,
                             len_seed=len_seed))


def listed():
    return [
        # a decode step of 256 sequences, some of which have ended (their pages go back): latency
        _plan('plan_decode_b256', 256, 1, 8192, 1, 64, 0.05, 0.05, 1),
        # the prompts of 16 sequences, small pages: about 70,000 slots
        _plan('plan_prompts_16seq', 16, 512, 8192, 0, 16, 0.0, 0.0, 2),
        # one sequence with four drafted tokens, a small vocabulary: latency
        _verify('verify_b1', 1, 5, 5, 32000, True, 'f32', 3),
        # 256 sequences with four drafted tokens each, draft and target probabilities in float32
        _verify('verify_b256', 256, 5, 5, 131072, True, 'f32', 4),
        # drafts looked up in the text itself (no draft probabilities), ragged, an odd vocabulary
        _verify('verify_lookup_bf16', 48, 1, 8, 50021, False, 'bf16', 5),
        # the decode step of 256 sequences: one new token each, q beside it
        _append('append4_decode_b256', 256, 1, 128, 1, 16, 2, 256, 64, False, True, 64, 'bf16', 6),
        # the prompts of 16 sequences (new = 0: all of each sequence is new) into small pages
        _append('append4_prompts_16seq', 16, 64, 512, 0, 32, 8, 128, 128, False, True, 16, 'bf16', 7),
        # the cached part of 16 prompts as dense keys and values, for the attention of their next part
        _read('read4_16seq', 16, 512, 8192, 8, 128, 16, 'bf16', 8),
        # one short chat turn: latency
        _attn('attn4_b1_short', 1, 77, 77, 1, 16, 2, 256, 16, True, 9),
        # 256 sequences of ordinary lengths: the throughput case, about 1.3 GB of cache
        _attn('attn4_b256', 256, 512, 8192, 1, 32, 8, 128, 64, False, 10),
        # one 131072-token context, two kv heads: everything hangs on the split over the length
        _attn('attn4_b1_131072', 1, 131072, 131072, 1, 16, 2, 256, 64, True, 11),
        # draft + verify: five new tokens of 16 ragged sequences, empty slots of a padded batch among them, pages
        # that divide no tile
        _attn('attn4_verify_16seq', 16, 0, 8192, 5, 24, 8, 64, 24, True, 12),
    ]


_MOST = 256 * 8192 * 8 * 128          # cache elements (padded to the longest sequence) of attn4_b256
_MOST_PROBS = 1280 * 131072           # target probabilities of verify_b256


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(['plan', 'verify', 'append', 'read', 'attn', 'attn'])
    seed = rng.randrange(1 << 20)
    if op == 'plan':
        seqs = _log_int(rng, 1, 4096)
        page = rng.choice([1, 8, 16, 20, 48, 64, 128, 256])
        gone, idle = rng.choice([0.0, 0.02, 0.2]), rng.choice([0.0, 0.1, 0.5])
        if rng.random() < 0.4:                        # prompts
            hi = _log_int(rng, 1, max(1, 131072 // seqs))
            return _plan(None, seqs, max(1, hi // 16), hi, 0, page, 0.0, idle, seed)
        return _plan(None, seqs, rng.choice([0, 1]), _log_int(rng, 1, 16384 if seqs <= 512 else 2048),
                     _log_int(rng, 1, 16), page, gone, idle, seed)
    if op == 'verify':
        vocab = _log_int(rng, 1000, 262144)
        if rng.random() < 0.5:
            vocab = max(64, vocab // 64 * 64)
        hi = rng.choice([1, 2, 3, 5, 8, 17])
        seqs = _log_int(rng, 1, max(1, min(512, _MOST_PROBS // (vocab * hi))))
        return _verify(None, seqs, rng.choice([0, 1, hi]), hi, vocab, rng.random() < 0.6, rng.choice(['f32', 'f32', 'bf16']),
                       seed)
    d = rng.choice([64, 128, 256])
    nkv = rng.choice([1, 2, 3, 4, 8])
    nq = nkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 16])
    page = rng.choice([1, 8, 16, 20, 32, 48, 64, 128, 256])
    dtype = rng.choice(['bf16', 'bf16', 'bf16', 'f32'])
    if op == 'append':
        rot = rng.choice([x for x in (0, 16, 32, 64, 96, 128, 256) if x <= d])
        seqs = _log_int(rng, 1, 256)
        new = rng.choice([1, 1, 2, 3, 5, 0])
        hi = _log_int(rng, 8, 512 if seqs <= 16 else 128)
        return _append(None, seqs, max(1, new), hi, new, nq, nkv, d, rot, rng.random() < 0.3, rng.random() < 0.8, page,
                       dtype, seed)
    if op == 'read':
        seqs = _log_int(rng, 1, 256)
        hi = _log_int(rng, 1, min(131072, 131072 * 1024 // (seqs * nkv * d)))
        return _read(None, seqs, rng.choice([0 if seqs > 8 else 1, max(1, hi // 16), hi]), hi, nkv, d, page, dtype, seed)
    seqs = _log_int(rng, 1, 256)
    new = rng.choice([1, 1, 1, 2, 3, 4, 6])
    most = min(131072, _MOST // (seqs * nkv * d) // max(1, nq * new // (8 * nkv)))
    hi = max(new, _log_int(rng, 16, max(16, most)))
    return _attn(None, seqs, rng.choice([0, hi // 16, hi]), hi, new, nq, nkv, d, page, rng.random() < 0.5, seed)


# ------------------------------------------------------------------------------- the inputs

_DT = {'bf16': torch.bfloat16, 'f32': torch.float32}


def _lens(case):
    """Cached lengths (the call's tokens included); a drawn length below the new tokens' count is an empty slot."""
    r = random.Random(case['len_seed'])
    n = [r.randint(case['lo'], case['hi']) for _ in range(case['seqs'])]
    return [x if x >= case['new'] else 0 for x in n]


def _requests(case):
    """Of each sequence: cached tokens, pages held, new tokens (-1: it has ended, its pages go back)."""
    r = random.Random(case['len_seed'])
    out = []
    for _ in range(case['seqs']):
        n, x, spare = r.randint(case['lo'], case['hi']), r.random(), r.random() < 0.2
        new = -1 if x < case['gone'] else 0 if x < case['gone'] + case['idle'] else case['new'] or n
        cached = n if case['new'] else 0
        # after refused drafts a sequence may hold a page more than its tokens need
        out.append((cached, (cached + case['page'] - 1) // case['page'] + (1 if spare and cached else 0), new))
    return out


def _rows(case):
    """Rows (tokens fed to the target) of each sequence of a verify case; one at least in all."""
    r = random.Random(case['len_seed'])
    n = [r.randint(case['lo'], case['hi']) for _ in range(case['seqs'])]
    return n if sum(n) else [1] + n[1:]


def _starts(lengths):
    return [0] + list(itertools.accumulate(lengths))


def _table(positions, rot, device):
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    ang = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * (1e6 ** (-2.0 * i / rot))
    return torch.cat([ang.cos(), ang.sin()], 1).to(torch.float32)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device='cuda')


def _prepare_plan(case, gen):
    req = _requests(case)
    P = case['page']
    held = [h for _, h, _ in req]
    after = [c + max(n, 0) for c, _, n in req]
    width = max(1, max(max(h, (a + P - 1) // P) for h, a in zip(held, after)))
    missing = sum(max(0, (a + P - 1) // P - h) for h, a, (_, _, n) in zip(held, after, req) if n > 0)
    spare = 7
    pages = sum(held) + missing + spare
    ids = torch.randperm(pages, generator=gen, device='cuda').to(torch.int32)
    H = _i32(held)
    col = torch.arange(width, device='cuda')
    start = H.long().cumsum(0) - H
    bt = torch.where(col < H[:, None], ids[(start[:, None] + col).clamp_max(pages - 1)], torch.zeros_like(ids[:1]))
    # the ring of free pages: `count` ids from position `head`, round its end; the rest of it is stale
    count, head = missing + spare, random.Random(case['len_seed']).randrange(pages)
    ring = torch.zeros(pages, dtype=torch.int32, device='cuda')
    ring[(head + torch.arange(count, device='cuda')) % pages] = ids[sum(held):]
    return dict(case=case, new=_i32([n for _, _, n in req]), lens=_i32([c for c, _, _ in req]), held=H,
                ring=_i32([head, count]), free=ring, bt=bt.contiguous(), T=sum(max(n, 0) for _, _, n in req))


def _prepare_verify(case, gen):
    rows, V, dt = _rows(case), case['vocab'], _DT[case['dtype']]
    cu = _starts(rows)
    T = cu[-1]
    even = len(set(rows)) == 1
    logits = torch.randn(T, V, generator=gen, device='cuda') * 3.0
    first = torch.zeros(T, dtype=torch.bool, device='cuda')
    last = torch.zeros(T, dtype=torch.bool, device='cuda')
    first[[a for a, n in zip(cu, rows) if n]] = True
    last[[a + n - 1 for a, n in zip(cu, rows) if n]] = True
    tokens = torch.randint(V, (T,), generator=gen, device='cuda', dtype=torch.int32)
    st = dict(case=case, cu=None if even else _i32(cu), uniform=torch.rand(T, generator=gen, device='cuda'), q=None,
              lens=torch.randint(64, 4096, (len(rows),), generator=gen, device='cuda', dtype=torch.int32))
    K = max(rows) - 1
    if case['draft'] and K:
        # the draft model's probabilities [sequences, drafts, vocabulary]: the target's, less sure; its tokens are
        # drawn from them (a sequence with fewer drafts leaves rows unused)
        d = torch.randn(len(rows), K, V, generator=gen, device='cuda').mul_(0.7)
        some = torch.arange(K, device='cuda') < _i32(rows)[:, None] - 1
        d[some] += logits[~last]
        st['q'] = torch.softmax(d, -1).to(dt)
        tokens[~first] = torch.multinomial(st['q'][some].float(), 1, generator=gen)[:, 0].to(torch.int32)
    elif K:
        guess = logits[~last].argmax(-1).to(torch.int32)
        tokens[~first] = torch.where(torch.rand(guess.shape, generator=gen, device='cuda') < 0.8, guess, tokens[~first])
        logits[~last, tokens[~first].long()] += 10.0                      # a text that repeats itself: likely tokens
    st.update(p=torch.softmax(logits, -1).to(dt), tokens=tokens)
    return st


def _quantised(gen, pages, nkv, P, d):
    """A cache of normal keys or values, by pages so that little float32 is held at a time."""
    c = torch.empty(pages, nkv, P, d // 2, dtype=torch.uint8, device='cuda')
    s = torch.empty(pages, nkv, P, d // GROUP, 2, dtype=torch.bfloat16, device='cuda')
    step = max(1, (1 << 28) // (nkv * P * d))
    for a in range(0, pages, step):
        x = torch.randn(min(step, pages - a), nkv, P, d, generator=gen, device='cuda')
        c[a:a + step], s[a:a + step] = _quantise(x)
    return c, s


def prepare(case, seed):
    dev = torch.device('cuda')
    gen = torch.Generator(device=dev).manual_seed(seed)
    if case['op'] == 'plan':
        return _prepare_plan(case, gen)
    if case['op'] == 'verify':
        return _prepare_verify(case, gen)
    dt = _DT[case.get('dtype', 'bf16')]

    def normal(*shape, std=1.0):
        x = torch.randn(*shape, generator=gen, device=dev, dtype=dt)
        return x if std == 1.0 else x.mul_(std)

    nkv, d, P = case['nkv'], case['d'], case['page']
    lens = _lens(case)
    width = max(1, max((n + P - 1) // P for n in lens))
    pages = sum((n + P - 1) // P for n in lens) + 3
    ids = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    at, rows = 0, []
    for n in lens:
        m = (n + P - 1) // P
        rows.append(torch.nn.functional.pad(ids[at:at + m], (0, width - m)))
        at += m
    st = dict(case=case, dt=dt, bt=torch.stack(rows), lens=_i32(lens))
    st['kc'], st['ks'] = _quantised(gen, pages, nkv, P, d)
    st['vc'], st['vs'] = _quantised(gen, pages, nkv, P, d)
    if case['op'] == 'read':
        st.update(T=sum(lens), cu=_i32(_starts(lens)))
    elif case['op'] == 'append':
        cu = _starts([case['new'] or n for n in lens])
        T = cu[-1]
        st.update(q=normal(T, case['nq'], d, std=2.0), k=normal(T, nkv, d, std=2.0), v=normal(T, nkv, d), T=T,
                  cu=None if case['new'] else _i32(cu), q_w=None, k_w=None,
                  table=_table(max(lens), case['rot'], dev) if case['rot'] else None)
        if case['norm']:
            st['q_w'], st['k_w'] = 1.0 + 0.1 * torch.randn(2, d, generator=gen, device=dev)
    else:
        T = case['seqs'] * case['new']
        st.update(q=normal(T, case['nq'], d, std=1.5), gate=normal(T, case['nq'], d) if case['gate'] else None)
    return st


# ------------------------------------------------------------------------------- the plain forms

def _plan_plain(st):
    case = st['case']
    N, P, T, cap = case['seqs'], case['page'], st['T'], st['free'].numel()
    new, lens, held = st['new'].long(), st['lens'].long(), st['held'].long()
    head, count = st['ring'].long()
    gone, add = new < 0, new.clamp_min(0)
    after = torch.where(gone, 0, lens + add)
    need = torch.where(add > 0, (after + P - 1) // P, 0)
    take = (need - held).clamp_min(0)
    end = take.cumsum(0)
    col = torch.arange(st['bt'].shape[1], device='cuda')
    fresh = (col >= held[:, None]) & (col < need[:, None])
    at = (head + (end - take)[:, None] + col - held[:, None]) % cap
    given = torch.where(gone[:, None] & (col < held[:, None]), st['bt'], -1)   # the pages that go back, in order
    st['bt'].copy_(torch.where(fresh, st['free'][at], st['bt']))
    back = torch.where(gone, held, 0)
    back_end = back.cumsum(0)
    ring_at = (head + count + (back_end - back)[:, None] + col) % cap
    # elsewhere the ring keeps what it held: those entries are sent behind its end
    buf = torch.cat([st['free'], st['free'][:1]])
    buf[torch.where(given >= 0, ring_at, cap)] = given.to(torch.int32)
    st['free'].copy_(buf[:cap])
    cu = torch.cat([add.new_zeros(1), add.cumsum(0)])
    t = torch.arange(T, device='cuda')
    s = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = lens[s] + t - cu[s]
    slot = st['bt'][s, pos // P].long() * P + pos % P
    out = torch.stack([(head + end[-1]) % cap, count - end[-1] + back_end[-1]])
    i32 = torch.int32
    return (cu.to(i32), pos.to(i32), slot, after.to(i32), torch.where(gone, 0, torch.maximum(held, need)).to(i32),
            out.to(i32), st['bt'], st['free'])


def _units(x):
    """Probabilities as whole multiples of 2^-42."""
    return torch.round(x.double().clamp(0.0, 1.0) * 2.0 ** 42).long()


def _verify_plain(st):
    case, p, q, tok, u = st['case'], st['p'], st['q'], st['tokens'].long(), st['uniform']
    N, T = case['seqs'], tok.shape[0]
    if st['cu'] is None:
        cu = torch.arange(N + 1, device='cuda') * (T // N)
    else:
        cu = st['cu'].long()
    bos, n = cu[:-1], cu[1:] - cu[:-1]
    t = torch.arange(T, device='cuda')
    s = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    i = t - bos[s]
    draft = tok[(t + 1).clamp_max(T - 1)]
    is_draft = i < n[s] - 1
    px = p[t, draft].double()
    if q is None:
        qx = torch.ones_like(px)
    else:
        qx = q[s, i.clamp_max(q.shape[1] - 1), draft].double()
    stop = ~(is_draft & (u.double() * qx < px))                   # the last row of a sequence always stops
    where = torch.where(stop, i, T)
    first = torch.full((N,), T, dtype=torch.int64, device='cuda').scatter_reduce(0, s, where, 'amin')
    some = n > 0
    acc = torch.where(some, first, 0)
    row = (bos + acc).clamp_max(T - 1)
    w = _units(p[row])
    refused = some & (acc < n - 1)
    if q is None:
        w[torch.arange(N, device='cuda'), draft[row]] *= (~refused).long()
    else:
        w = (w - _units(q[torch.arange(N, device='cuda'), acc.clamp_max(q.shape[1] - 1)]) * refused[:, None]).clamp_min(0)
    empty = refused & (w.sum(-1) == 0)                            # nothing is left of p: drawn from p itself
    w = torch.where(empty[:, None], _units(p[row]), w)
    c = w.cumsum(-1)
    # the number of a sequence's last row draws the token: the first with C 2^24 > U W
    U = torch.floor(u[(cu[1:] - 1).clamp_min(0)].double() * 2.0 ** 24).long()
    W = c[:, -1]
    level = (W >> 24) * U + (((W & 0xffffff) * U) >> 24)
    drawn = (c <= level[:, None]).sum(-1)
    out = torch.where(i < acc[s], draft, torch.where(i == acc[s], drawn[s], -1))
    return acc.to(torch.int32), out.to(torch.int32), (st['lens'] - torch.where(some, n - 1 - acc, 0)).to(torch.int32)


def _quantise(x):
    """float32 [..., d] -> bytes [..., d/2], scales [..., d/64, 2]."""
    g = x.unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    # quotients of short numbers meet borders: true divisions (by a tensor), halves to even
    s = ((hi - lo) / torch.full_like(lo, 15.0)).bfloat16()
    m = lo.bfloat16()
    n = ((g - m.float()) / torch.where(s > 0, s.float(), math.inf)).round_().clamp_(0.0, 15.0).to(torch.uint8).flatten(-2)
    return n[..., 0::2] | (n[..., 1::2] << 4), torch.cat([s, m], -1)


def _values(c, s):
    """Bytes [..., d/2] and scales [..., d/64, 2] -> float32 [..., d]."""
    n = torch.stack([c & 15, c >> 4], -1).flatten(-2).unflatten(-1, (-1, GROUP)).float()
    s = s.float()
    return (n * s[..., :1] + s[..., 1:]).flatten(-2)


def _norm_rope_plain(x, w, cs, inter):
    """x [T, H, D] -> float32; w [D] or None; cs [T, r] or None (the table rows of the tokens)."""
    u = x.float()
    if w is not None:
        u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + 1e-6) * w
    if cs is None:
        return u
    r = cs.shape[1]
    c, s = cs[:, None, :r // 2], cs[:, None, r // 2:]
    if inter:
        a, b = u[..., 0:r:2], u[..., 1:r:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = u[..., :r // 2], u[..., r // 2:r]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, u[..., r:]], -1)


def _places(st):
    """Page and slot of each new token (of all of a sequence where new = 0), and its index in the cache."""
    case = st['case']
    t = torch.arange(st['T'], device='cuda')
    if st['cu'] is None:
        s, i = t // case['new'], t % case['new']
        new = case['new']
    else:
        s = torch.searchsorted(st['cu'][1:].contiguous(), t, right=True)
        i = t - st['cu'][s]
        new = st['lens'][s]
    pos = (st['lens'][s] - new + i).long()
    return st['bt'][s, pos // case['page']].long(), pos % case['page'], pos, st['lens'][s] > 0


def _read_plain(st):
    page, slot, _, some = _places(st)
    k, v = (_values(st[c][page, :, slot], st[s][page, :, slot]) for c, s in (('kc', 'ks'), ('vc', 'vs')))
    return k.to(st['dt']), v.to(st['dt'])


def _append_plain(st):
    case = st['case']
    page, slot, pos, some = _places(st)
    cs = st['table'][pos.clamp_min(0)] if st['table'] is not None else None
    k = _norm_rope_plain(st['k'], st['k_w'], cs, case['inter'])
    for x, c, s in ((k, 'kc', 'ks'), (st['v'].float(), 'vc', 'vs')):
        st[c][page, :, slot], st[s][page, :, slot] = _quantise(x)
    return (_norm_rope_plain(st['q'], st['q_w'], cs, case['inter']).to(st['dt']),) + _read_plain(st)


def _attn_plain(st):
    case = st['case']
    N, n, nkv, d, P = case['seqs'], case['new'], case['nkv'], case['d'], case['page']
    G = case['nq'] // nkv
    L = st['bt'].shape[1] * P
    bt = st['bt'].long()
    K = _values(st['kc'][bt], st['ks'][bt]).transpose(1, 2).reshape(N, nkv, L, d)
    q = st['q'].float().reshape(N, n, nkv, G, d).transpose(1, 2).reshape(N, nkv, n * G, d)
    sc = (q @ K.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).reshape(N, nkv, n, G, L)
    del K
    # token i of n sees the cache indices up to len - n + i
    limit = st['lens'][:, None] - n + torch.arange(n, device='cuda')
    seen = torch.arange(L, device='cuda') <= limit[..., None]
    sc.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = sc.amax(-1, keepdim=True).clamp_min(-1e30)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    V = _values(st['vc'][bt], st['vs'][bt]).transpose(1, 2).reshape(N, nkv, L, d)
    o = p.reshape(N, nkv, n * G, L) @ V
    del V
    o = o.reshape(N, nkv, n, G, d) / l.clamp_min(1e-30)
    o = o.transpose(1, 2).reshape(N * n, nkv * G, d)
    if st['gate'] is not None:
        o = o * torch.sigmoid(st['gate'].float())
    return o.to(st['dt'])


# ------------------------------------------------------------------------------- one pass

def run(st):
    case = st['case']
    if not own:
        return {'plan': _plan_plain, 'verify': _verify_plain, 'append': _append_plain, 'read': _read_plain,
                'attn': _attn_plain}[case['op']](st)
    from gated_deltanet_linear_conv_gb300 import gdn
    if case['op'] == 'plan':
        p = gdn.paged_plan(st['new'], st['lens'], st['held'], st['ring'], st['free'], st['bt'], case['page'], st['T'])
        return p.cu_seqlens, p.positions, p.slots, p.kv_lens, p.pages_held, p.free_ring, st['bt'], st['free']
    if case['op'] == 'verify':
        return gdn.draft_verify(st['p'], st['tokens'], st['uniform'], st['q'], cu_seqlens=st['cu'], num_seqs=case['seqs'],
                                kv_lens=st['lens'])
    cache = (st['kc'], st['vc'], st['ks'], st['vs'], st['bt'], st['lens'])
    if case['op'] == 'attn':
        return gdn.paged_kv4_attn_decode(st['q'], *cache, gate=st['gate'])
    q = ()
    if case['op'] == 'append':
        q = (gdn.paged_kv4_append(st['k'], st['v'], *cache, q=st['q'], cos_sin=st['table'], q_norm_w=st['q_w'],
                                  k_norm_w=st['k_w'], cu_seqlens=st['cu'], interleaved=case['inter'],
                                  out_dtype=st['dt']),)
    return q + gdn.paged_kv4_read(*cache, st['T'], cu_seqlens=st['cu'], out_dtype=st['dt'])


# ------------------------------------------------------------------------------- work and 64-bit values

def work(case):
    if case['op'] == 'plan':
        req, P = _requests(case), case['page']
        T = sum(max(n, 0) for _, _, n in req)
        moved = sum(max(0, (c + n + P - 1) // P - h) if n > 0 else h if n < 0 else 0 for c, h, n in req)
        # lengths, requests and pages held in, lengths, pages held and bounds out; a table entry or more per request
        return dict(bytes=7 * 4 * case['seqs'] + 12 * T + 8 * moved, flops=8.0 * T)
    if case['op'] == 'verify':
        es = 2 if case['dtype'] == 'bf16' else 4
        # the target's row that draws, and the draft's where a token was refused (about seven of ten sequences)
        some = sum(n > 0 for n in _rows(case))
        rows = some * (1.7 if case['draft'] and case['hi'] > 1 else 1.0)
        return dict(bytes=int(rows * case['vocab'] * es) + 16 * sum(_rows(case)), flops=4.0 * rows * case['vocab'])
    es = 4 if case.get('dtype') == 'f32' else 2
    nkv, d = case['nkv'], case['d']
    lens = _lens(case)
    held = nkv * d * 9 // 16                           # bytes of a token's keys (or values): 4.5 bits an element
    if case['op'] == 'read':
        return dict(bytes=2 * sum(lens) * (held + nkv * d * es) + 4 * sum(lens) // case['page'],
                    flops=4.0 * sum(lens) * nkv * d)
    nq = case['nq']
    if case['op'] == 'append':
        T = sum(case['new'] or n for n in lens)
        return dict(bytes=T * (2 * nq * d * es + 4 * nkv * d * es + 2 * held) + 4 * min(T, max(lens)) * case['rot'] + 4 * T,
                    flops=T * (10.0 * nq * d + 30.0 * nkv * d))
    T = case['seqs'] * case['new']
    return dict(bytes=2 * sum(lens) * held + (3 if case['gate'] else 2) * T * nq * d * 2 + 4 * sum(lens) // case['page'],
                flops=4.0 * sum(lens) * case['new'] * nq * d)


def _plan_exact(case, st):
    """Request by request on the host."""
    req, P, cap = _requests(case), case['page'], st['free'].numel()
    bt, free = st['bt'].tolist(), st['free'].tolist()
    head, count = st['ring'].tolist()
    taken, cu, pos, slot, lens, held = 0, [0], [], [], [], []
    back = []
    for s, (cached, h, n) in enumerate(req):
        if n < 0:
            back += bt[s][:h]
            lens.append(0)
            held.append(0)
        else:
            while n > 0 and h * P < cached + n:
                bt[s][h] = free[(head + taken) % cap]
                taken += 1
                h += 1
            for x in range(cached, cached + n):
                pos.append(x)
                slot.append(bt[s][x // P] * P + x % P)
            lens.append(cached + n)
            held.append(h)
        cu.append(cu[-1] + max(n, 0))
    for r, page in enumerate(back):
        free[(head + count + r) % cap] = page
    ring = [(head + taken) % cap, count - taken + len(back)]
    return (_i32(cu), _i32(pos), torch.tensor(slot, dtype=torch.int64, device='cuda'), _i32(lens), _i32(held), _i32(ring),
            _i32(bt), _i32(free))


def _verify_exact(case, st):
    """Sequence by sequence: Python's whole numbers and bisection."""
    rows = _rows(case)
    tok, u = st['tokens'].tolist(), st['uniform'].tolist()
    acc, out, lens, t = [], [], st['lens'].tolist(), 0
    for s, n in enumerate(rows):
        if n == 0:
            acc.append(0)
            continue
        a = 0
        while a < n - 1:
            x = tok[t + a + 1]
            q = 1.0 if st['q'] is None else float(st['q'][s, a, x])
            if not u[t + a] * q < float(st['p'][t + a, x]):
                break
            a += 1
        w = [int(x) for x in (st['p'][t + a].double() * 2.0 ** 42).round().tolist()]
        if a < n - 1:
            if st['q'] is None:
                w[tok[t + a + 1]] = 0
            else:
                w = [max(0, x - int(y)) for x, y in zip(w, (st['q'][s, a].double() * 2.0 ** 42).round().tolist())]
            if not any(w):
                w = [int(x) for x in (st['p'][t + a].double() * 2.0 ** 42).round().tolist()]
        c = list(itertools.accumulate(w))
        drawn = bisect.bisect_right(c, (int(u[t + n - 1] * 2 ** 24) * c[-1]) >> 24)
        acc.append(a)
        out += tok[t + 1:t + 1 + a] + [drawn] + [-1] * (n - 1 - a)
        lens[s] -= n - 1 - a
        t += n
    return _i32(acc), _i32(out), _i32(lens)


def _exact_rows(x, w, pos, table, inter):
    """One row set in 64 bits: complex multiplication by cos + i sin of each pair."""
    u = x.double()
    if w is not None:
        u = u / (u.pow(2).sum(-1, keepdim=True) / u.shape[-1] + 1e-6).sqrt() * w.double()
    if table is None:
        return u
    h = table.shape[1] // 2
    rot = torch.complex(table[pos, :h].double(), table[pos, h:].double()).unsqueeze(1)
    out = u.clone()
    if inter:
        z = torch.view_as_complex(u[..., :2 * h].reshape(*u.shape[:-1], h, 2).contiguous()) * rot
        out[..., :2 * h] = torch.view_as_real(z).reshape(*u.shape[:-1], 2 * h)
    else:
        z = torch.complex(u[..., :h], u[..., h:2 * h]) * rot
        out[..., :h], out[..., h:2 * h] = z.real, z.imag
    return out


def _held_exact(x):
    """What 4 bits hold of x: its groups one after another."""
    out = torch.empty_like(x)
    for a in range(0, x.shape[-1], GROUP):
        g = x[..., a:a + GROUP]
        least = g.min(-1, keepdim=True).values
        step = ((g.max(-1, keepdim=True).values - least) / 15.0).bfloat16().double()
        base = least.bfloat16().double()
        n = torch.round((g - base) / torch.where(step > 0, step, 1.0)).clamp(0, 15)
        out[..., a:a + GROUP] = base + n * step
    return out


def _dense_exact(c, s):
    """A cache's bytes and scales as values in 64 bits."""
    out = torch.empty(*c.shape[:-1], 2 * c.shape[-1], dtype=torch.float64, device=c.device)
    out[..., 0::2], out[..., 1::2] = (c % 16).double(), torch.div(c, 16, rounding_mode='floor').double()
    s = s.double().repeat_interleave(GROUP, -2)
    return out * s[..., 0] + s[..., 1]


def exact(case, seed):
    if case['op'] == 'attn' and work(case)['flops'] > 4e12:
        return None                                   # over 20 seconds of 64-bit products
    if case['op'] == 'verify' and case['seqs'] * case['vocab'] > 5e6:
        return None                                   # over 20 seconds of Python's whole numbers
    st = prepare(case, seed)
    if case['op'] == 'plan':
        return _plan_exact(case, st)
    if case['op'] == 'verify':
        return _verify_exact(case, st)
    lens, P = _lens(case), case['page']
    bt = st['bt'].tolist()
    if case['op'] in ('append', 'read'):
        where = [(s, p) for s, n in enumerate(lens) for p in range(n - (case['new'] or n), n)]
        pos = torch.tensor([p for _, p in where], dtype=torch.int64, device='cuda')
        page = torch.tensor([bt[s][p // P] for s, p in where], dtype=torch.int64, device='cuda')
        if case['op'] == 'read':
            return tuple(_dense_exact(st[c][page, :, pos % P], st[s][page, :, pos % P])
                         for c, s in (('kc', 'ks'), ('vc', 'vs')))
        q, k = (_exact_rows(st[x], st[x + '_w'], pos, st['table'], case['inter']) for x in 'qk')
        return q, _held_exact(k), _held_exact(st['v'].double())
    n, G, d = case['new'], case['nq'] // case['nkv'], case['d']
    out = torch.zeros(case['seqs'] * n, case['nq'], d, dtype=torch.float64, device='cuda')
    for s, L in enumerate(lens):
        if L == 0:
            continue
        pages = st['bt'][s, :(L + P - 1) // P].long()
        for h in range(case['nkv']):
            K = _dense_exact(st['kc'][pages, h], st['ks'][pages, h]).reshape(-1, d)[:L]
            V = _dense_exact(st['vc'][pages, h], st['vs'][pages, h]).reshape(-1, d)[:L]
            for i in range(n):
                e = L - n + i + 1
                q = st['q'][s * n + i, h * G:(h + 1) * G].double()
                a = torch.softmax(q @ K[:e].T / math.sqrt(d), -1)
                out[s * n + i, h * G:(h + 1) * G] = a @ V[:e]
    if st['gate'] is not None:
        out = out / (1.0 + torch.exp(-st['gate'].double()))
    return out
