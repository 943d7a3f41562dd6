"""Beam search's selection and reordering on the GPU against plain references
in 64 bits, and a whole search on the decoder."""
import math

import numpy as np
import pytest
import torch

from persistent_megakernel_03_b200 import binding, synth
from kv4_util import Plain

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _reference(logits, cum, finished, eos):
    """logits [n][W][V] float64 -> tokens, parents, scores, done, and the
    smallest gap between scores of different beams that decides something."""
    n, W, V = logits.shape
    out = [[], [], [], []]
    for b in range(n):
        found = []
        for w in range(W):
            if finished[b, w]:
                if cum[b, w] > -np.inf:
                    found.append((-cum[b, w], w, 0, 0, eos))
                continue
            x = logits[b, w]
            if np.isnan(x).any() or (x == np.inf).any() or not (x > -np.inf).any():
                continue
            lse = x.max() + np.log(np.exp(x - x.max()).sum())
            order = np.argsort(-x, kind="stable")[:W]
            found += [(-(cum[b, w] + x[v] - lse), w, i, v, v) for i, v in enumerate(order)
                      if x[v] > -np.inf and cum[b, w] > -np.inf]
        found = sorted(found)[:W]
        found += [(np.inf, w, 0, 0, max(eos, 0)) for w in range(len(found), W)]
        out[0].append([f[4] for f in found])
        out[1].append([f[1] for f in found])
        out[2].append([-f[0] for f in found])
        out[3].append([bool(finished[b, f[1]]) or (eos >= 0 and f[4] == eos) for f in found])
    return [np.array(o) for o in out]


def _run(logits, cum, finished=None, eos=-1, done=True):
    n, W = cum.shape
    dev = "cuda"
    tok = torch.full((n, W), -9, dtype=torch.int32, device=dev)
    par, sc = torch.full_like(tok, -9), torch.full((n, W), 5.0, device=dev)
    fin = torch.full((n, W), 7, dtype=torch.uint8, device=dev) if done else None
    V = logits.shape[1]
    ws = torch.full((binding.beam_select_workspace_bytes(n, W, V),), 0xFF, dtype=torch.uint8, device=dev)
    binding.beam_select(logits, cum, tok, par, sc, ws, finished=finished, finished_out=fin, eos=eos)
    return tok, par, sc, fin


def _check(logits, cum, finished=None, eos=-1):
    tok, par, sc, fin = _run(logits, cum, finished, eos)
    n, W = cum.shape
    f = np.zeros((n, W), bool) if finished is None else finished.bool().cpu().numpy()
    want = _reference(logits.double().cpu().numpy().reshape(n, W, -1), cum.double().cpu().numpy(), f, eos)
    assert np.array_equal(tok.cpu().numpy(), want[0])
    assert np.array_equal(par.cpu().numpy(), want[1])
    got = sc.double().cpu().numpy()
    dead = np.isinf(want[2])
    assert np.array_equal(np.isinf(got), dead) and (got[dead] == -np.inf).all()
    # the sum of exponentials in fp32 (16 a thread, 5 + 3 pairwise additions, each
    # exponential 2^-22): 2^-18 on the logarithm; one rounding to fp32
    lim = np.abs(want[2][~dead]) * 2.0 ** -24 + 2.0 ** -18
    assert (np.abs(got[~dead] - want[2][~dead]) <= lim).all()
    assert np.array_equal(fin.cpu().numpy().astype(bool), want[3])


def _logits(rows, V, dtype, seed, size=3.0):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn(rows, V, generator=g)).to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,W,V", [
    (1, 1, 1), (1, 1, 2), (1, 4, 4096), (2, 4, 4097), (3, 2, 4095), (1, 8, 151936), (2, 16, 8191), (5, 3, 100),
    (1, 16, 16), (1, 8, 3), (16, 4, 1000), (1, 5, 70001), (1, 16, 1048576)])
def test_select_matches_the_reference(cuda_ok, dtype, n, W, V):
    x = _logits(n * W, V, TYPES[dtype], V + W).cuda()
    cum = (torch.rand(n, W, generator=torch.Generator().manual_seed(1)) * -2 - 5).cuda()
    _check(x, cum)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offset,extra", [(0, 8), (0, 1), (3, 13), (1, 0)])
def test_select_takes_strided_and_unaligned_rows(cuda_ok, dtype, offset, extra):
    V = 5003
    wide = _logits(8, V + offset + extra, TYPES[dtype], 5).cuda()
    cum = torch.zeros(2, 4, device="cuda") - torch.arange(8, device="cuda").view(2, 4)
    _check(wide[:, offset:offset + V], cum)


@pytest.mark.parametrize("dtype", TYPES)
def test_select_ties_go_to_the_lowest_beam_and_token(cuda_ok, dtype):
    """Equal rows, equal sums, few distinct logits: every order is by place."""
    x = torch.zeros(12, 9000, dtype=TYPES[dtype], device="cuda")
    _check(x, torch.zeros(3, 4, device="cuda"))
    row = torch.randint(0, 3, (1, 9000), generator=torch.Generator().manual_seed(2)).float()
    x = row.expand(12, 9000).contiguous().to(TYPES[dtype]).cuda()
    _check(x, torch.zeros(3, 4, device="cuda"))
    x = -x      # -0.0 beside 0.0 is a tie
    x[:, ::2] += 0.0
    _check(x, torch.zeros(3, 4, device="cuda"))


def test_select_masks_dead_and_finished_beams(cuda_ok):
    V, eos = 6000, 17
    x = _logits(24, V, torch.float32, 3)
    cum = torch.rand(4, 6, generator=torch.Generator().manual_seed(4)) * -3
    x[0:6] = -float("inf")                      # nothing allowed at all
    x[6:12] = -float("inf")
    x[7, 5999], x[9, 0], x[9, 4096] = 1.0, 2.0, 2.0    # three candidates for six beams
    cum[2, 1:] = -float("inf")                  # a first step: one live beam
    x[18] = float("nan")
    x[19, 7] = float("nan")
    x[20, 8] = float("inf")
    finished = torch.zeros(4, 6, dtype=torch.bool)
    finished[3, 3:5] = True
    finished[2, 2] = True                       # finished, and its sum is -inf
    cum[3, 3] = 0.5                             # best of all
    _check(x.cuda(), cum.cuda(), finished.cuda(), eos)
    _check(x.cuda(), cum.cuda())
    finished[:] = True
    _check(x.cuda(), cum.cuda(), finished.cuda(), eos)
    cum[:] = float("nan")
    tok, par, sc, fin = _run(x.cuda(), cum.cuda(), finished.cuda(), eos)
    assert (sc == -float("inf")).all() and torch.equal(par, torch.arange(6, device="cuda").expand(4, 6).int())


def test_select_masked_tail_and_extreme_logits(cuda_ok):
    x = _logits(4, 20000, torch.float32, 9, size=200.0)
    x[:, 13000:] = -float("inf")
    x[0, 0], x[1, 12999] = 3.0e38, -3.0e38
    _check(x.cuda(), torch.tensor([[0.0, -1.0, -2.0, -1000.0]]).cuda())


def _exact(logits, cum):
    """tokens and parents of the highest scores, each row's sum of exponentials
    rounded once (math.fsum: rows of the same logits in another order have the
    same), and the smallest distance of two scores of different beams that
    are not equal, among the W + 1 first."""
    n, W, V = logits.shape
    tok, par, gap = [], [], np.inf
    for b in range(n):
        found = []
        for w in range(W):
            x = logits[b, w]
            lse = x.max() + math.log(math.fsum(np.exp(x - x.max())))
            order = np.argsort(-x, kind="stable")[:W + 1]
            found += [(-(cum[b, w] + (x[v] - lse)), w, i, v) for i, v in enumerate(order)]
        found = sorted(found)[:W + 1]
        for f, g in zip(found, found[1:]):
            if f[1] != g[1] and f[0] != g[0]:
                gap = min(gap, g[0] - f[0])
        tok.append([f[3] for f in found[:W]])
        par.append([f[1] for f in found[:W]])
    return np.array(tok), np.array(par), gap


def _check_exact(logits, cum):
    tok, par, sc, _ = _run(logits, cum)
    n, W = cum.shape
    want = _exact(logits.double().cpu().numpy().reshape(n, W, -1), cum.double().cpu().numpy())
    assert want[2] > 1e-12          # far above what 64 bits lose
    assert np.array_equal(par.cpu().numpy(), want[1])
    assert np.array_equal(tok.cpu().numpy(), want[0])
    assert (sc[:, 1:] <= sc[:, :-1]).all()


def _shuffled(n, W, V, dtype, seed):
    """Rows of a search: one row's logits, each time in another order."""
    g = torch.Generator().manual_seed(seed)
    one = (3 * torch.randn(n, 1, V, generator=g)).to(dtype).expand(n, W, V)
    at = torch.rand(n, W, V, generator=g).argsort(-1)
    return one.gather(2, at).reshape(n * W, V).contiguous()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,W,V", [(6, 2, 9001), (4, 3, 40000), (3, 8, 30011), (1, 4, 151936), (2, 16, 5000)])
def test_select_equal_sums_of_shuffled_rows_go_to_the_lowest_beam(cuda_ok, dtype, n, W, V):
    """Equal sums and the same logits in another order: every score is a tie of
    all beams, whatever order a kernel adds in."""
    _check_exact(_shuffled(n, W, V, TYPES[dtype], V + W).cuda(), torch.full((n, W), -1.25, device="cuda"))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,W,V,step", [(8, 2, 9001, 1), (4, 4, 60000, 2), (2, 8, 30011, 3), (3, 16, 4097, 1), (1, 2, 151936, 1)])
def test_select_orders_beams_a_rounding_apart(cuda_ok, dtype, n, W, V, step):
    """Sums `step` fp32 numbers apart (6e-8 each), higher ones in random places."""
    x = _shuffled(n, W, V, TYPES[dtype], V)
    cum = np.full((n, W), np.float32(-0.75)).view(np.int32)
    rng = np.random.default_rng(W)
    cum = cum + step * np.stack([rng.permutation(W) for _ in range(n)]).astype(np.int32)
    _check_exact(x.cuda(), torch.from_numpy(cum.astype(np.int32).view(np.float32)).cuda())


def test_select_orders_beams_whose_sums_differ_in_the_tail(cuda_ok):
    """Same highest logits, sums of exponentials 3e-8 to 4e-7 apart by one logit
    far down; a finished beam whose sum lies in between."""
    n, W, V = 4, 4, 50000
    x = _shuffled(n, W, V, torch.float32, 5).view(n, W, V)
    rng = np.random.default_rng(5)
    for b in range(n):
        for w, k in enumerate(rng.permutation(W)):
            low = int(x[b, w].argmin())
            lse = float(torch.logsumexp(x[b, w].double(), 0))
            x[b, w, low] = lse + math.log(1e-7 * (k + 0.3))
    cum = torch.full((n, W), -2.0)
    _check_exact(x.reshape(n * W, V).cuda(), cum.cuda())
    # beam 2 has finished, its sum the fp32 number next to the best score of beam 0
    finished = torch.zeros(n, W, dtype=torch.bool)
    finished[:, 2] = True
    for b in range(n):
        best = float(x[b, 0].max().double() - torch.logsumexp(x[b, 0].double(), 0)) - 2.0
        cum[b, 2] = best
    flat = x.reshape(n * W, V)
    tok, par, sc, _ = _run(flat.cuda(), cum.cuda(), finished.cuda(), 9)
    want = _reference(flat.double().numpy().reshape(n, W, V), cum.double().numpy(), finished.numpy(), 9)
    assert np.array_equal(par.cpu().numpy(), want[1]) and np.array_equal(tok.cpu().numpy(), want[0])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,W,V", [(8, 4, 9001), (4, 8, 70000), (3, 16, 300)])
def test_select_rows_that_differ_by_a_constant_tie(cuda_ok, dtype, n, W, V):
    """A constant on all logits of a row changes no log-probability: with equal sums
    every score is a tie of all beams.  Multiples of 1/8 between -8 and 8 hold
    the shifts, of up to 8, exactly in every type."""
    x = (_shuffled(n, W, V, torch.float32, V).clamp(-8, 8) * 8).round() / 8
    shift = torch.randint(-32, 33, (n * W, 1), generator=torch.Generator().manual_seed(W)).float() / 4
    x = (x + shift).to(TYPES[dtype])
    assert torch.equal(x.double().frac().mul(8).frac(), torch.zeros_like(x.double()))
    tok, par, sc, _ = _run(x.cuda(), torch.full((n, W), -0.7, device="cuda"))
    x = x.double().numpy().reshape(n, W, V)
    for b in range(n):
        level = x[b] - x[b].max(-1, keepdims=True)
        order = sorted((-level[w, v], w, i, v) for w in range(W)
                       for i, v in enumerate(np.argsort(-level[w], kind="stable")[:W]))[:W]
        assert par[b].tolist() == [o[1] for o in order]
        assert tok[b].tolist() == [o[3] for o in order]


def test_select_close_beams_replayed_and_repeated(cuda_ok):
    """The same bits from a graph and from every call, also where beams are close."""
    x = _shuffled(4, 4, 20000, torch.float16, 3).cuda()
    cum = torch.full((4, 4), -3.0, device="cuda")
    first = _run(x, cum)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, _run(x, cum)))
    tok = torch.zeros(4, 4, dtype=torch.int32, device="cuda")
    par, sc = torch.zeros_like(tok), torch.zeros(4, 4, device="cuda")
    ws = torch.empty(binding.beam_select_workspace_bytes(4, 4, 20000), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.beam_select(x, cum, tok, par, sc, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first[:3], (tok, par, sc)))


def test_select_without_finished_flags_out(cuda_ok):
    x = _logits(4, 300, torch.float32, 1).cuda()
    cum = torch.zeros(1, 4, device="cuda")
    a, b = _run(x, cum, done=False), _run(x, cum)
    assert all(torch.equal(p, q) for p, q in zip(a[:3], b[:3]))


def test_select_two_at_once_and_replayed(cuda_ok):
    x = [_logits(8, 30000, torch.bfloat16, s).cuda() for s in (1, 2)]
    cum = torch.zeros(2, 4, device="cuda")
    one = [_run(v, cum) for v in x]
    streams = [torch.cuda.Stream() for _ in x]
    torch.cuda.synchronize()
    both = []
    for v, st in zip(x, streams):
        with torch.cuda.stream(st):
            both.append(_run(v, cum))
    torch.cuda.synchronize()
    for a, b in zip(one, both):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    buf = x[0].clone()
    tok = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    par, sc = torch.zeros_like(tok), torch.zeros(2, 4, device="cuda")
    ws = torch.empty(binding.beam_select_workspace_bytes(2, 4, 30000), dtype=torch.uint8, device="cuda")
    state = torch.arange(8 * 3 * 5 * 8, device="cuda", dtype=torch.int32).view(8, 3, 5, 8)
    keep = state.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.beam_select(buf, cum, tok, par, sc, ws)
        binding.beam_reorder(state, par, 1, 4)
    for v, a in zip(x, one):
        buf.copy_(v)
        state.copy_(keep)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(tok, a[0]) and torch.equal(par, a[1]) and torch.equal(sc, a[2])
        rows = (par.long() + torch.tensor([[0], [4]], device="cuda")).flatten()
        want = keep.clone()
        want[:, :, 1:] = keep[rows][:, :, 1:]
        assert torch.equal(state, want)


# ----------------------------------------------------------------- reorder

def _parents(n, W, kind, seed=0):
    rng = np.random.default_rng(seed)
    p = {"identity": np.tile(np.arange(W), (n, 1)), "cycle": np.tile((np.arange(W) + 1) % W, (n, 1)),
         "one": np.full((n, W), W - 1), "random": rng.integers(0, W, (n, W)),
         "bad": rng.integers(-3, W + 3, (n, W))}[kind]
    return p.astype(np.int32)


@pytest.mark.parametrize("kind", ["identity", "cycle", "one", "random", "bad"])
@pytest.mark.parametrize("n,W,segs,pos,row,first,count", [
    (1, 1, 1, 1, 16, 0, 1), (1, 2, 1, 1, 16, 0, 1), (1, 2, 3, 5, 32, 2, 3), (3, 4, 16, 40, 128, 7, 33),
    (2, 5, 1000, 2, 16, 0, 1), (1, 8, 7, 300, 256, 0, 300), (4, 16, 3, 33, 48, 1, 31), (1, 9, 2, 4097, 16, 4, 4093)])
def test_reorder_moves_rows_in_place(cuda_ok, kind, n, W, segs, pos, row, first, count):
    rng = np.random.default_rng(3)
    state = rng.integers(0, 256, (n * W, segs, pos, row), dtype=np.uint8)
    par = _parents(n, W, kind, W)
    t = torch.from_numpy(state.copy()).cuda()
    binding.beam_reorder(t, torch.from_numpy(par).cuda(), first, count)
    src = np.where((par >= 0) & (par < W), par, np.arange(W))
    rows = (src + np.arange(n)[:, None] * W).reshape(-1)
    want = state.copy()
    want[:, :, first:first + count] = state[rows][:, :, first:first + count]
    assert np.array_equal(t.cpu().numpy(), want)


def test_reorder_of_segments_that_hold_all_beams(cuda_ok):
    """[layer][beam][...]: beams inside a segment."""
    W, layers, size = 4, 6, 96
    state = torch.randint(0, 255, (layers, W, size), dtype=torch.uint8)
    par = torch.tensor([[2, 2, 0, 1]], dtype=torch.int32)
    t = state.cuda()
    rc = binding.lib().mk_beam_reorder(t.data_ptr(), par.cuda().data_ptr(), 1, W, size, layers, W * size, size,
                                       torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert torch.equal(t.cpu(), state[:, par[0].long()])


def test_reorder_of_states_past_32_bits(cuda_ok):
    size = 1 << 30
    state = torch.zeros(3, 2, 1, size, dtype=torch.uint8, device="cuda")      # 6 GB
    for r in range(3):
        for i in range(2):
            state[r, i, 0, :64] = 10 * r + i
            state[r, i, 0, -64:] = 100 + 10 * r + i
    binding.beam_reorder(state, torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda"), 0, 1)
    for r, p in enumerate((2, 0, 1)):
        for i in range(2):
            assert (state[r, i, 0, :64] == 10 * p + i).all() and (state[r, i, 0, -64:] == 100 + 10 * p + i).all()


@pytest.mark.parametrize("dim,page,paged,scores", [(64, 32, True, True), (128, 96, True, False), (64, 128, False, True)])
def test_kv4_reorder_moves_blocks_and_scores(cuda_ok, dim, page, paged, scores):
    n, W, heads, per = 2, 3, 2, 3
    p = Plain(n * W, heads, dim, page, per, seed=4, n_pages=n * W * per + (2 if paged else 0))
    if not paged:
        p.table = np.arange(n * W * per).reshape(n * W, per).astype(np.int32)
    p.pool[:] = np.random.default_rng(1).integers(0, 256, p.pool.shape)
    if paged:
        p.table[:3, 0] = p.table[0, 0]       # a search's beams share their prompt's page
        p.table[4, 2] = -1
    sc = np.random.default_rng(2).normal(size=(n * W, heads, p.capacity)).astype(np.float32)
    cache = binding.Kv4Cache(torch.from_numpy(p.pool.copy()).cuda(), torch.zeros(n * W, dtype=torch.int32, device="cuda"),
                             heads, dim, page, torch.from_numpy(p.table).cuda() if paged else None,
                             torch.from_numpy(sc.copy()).cuda() if scores else None)
    par = np.array([[1, 0, 0], [2, 2, 1]], np.int32)
    first, keys = page + 5, min(2 * page + 33, p.capacity)
    binding.kv4_reorder(cache, torch.from_numpy(par).cuda(), first, keys)
    b0, b1 = first // 32, -(-keys // 32)
    size = 32 * (dim + dim // 8)
    old = p.pool.copy().reshape(p.pool.shape[0], heads, page // 32, size)
    new = old.copy()
    want = sc.copy()
    for s in range(n):
        for w in range(W):
            a, b = s * W + par[s, w], s * W + w
            for blk in range(b0, b1):
                pa, pb = p.table[a, blk * 32 // page], p.table[b, blk * 32 // page]
                if pa >= 0 and pb >= 0:
                    new[pb, :, blk % (page // 32)] = old[pa, :, blk % (page // 32)]
            want[b, :, b0 * 32:b1 * 32] = sc[a, :, b0 * 32:b1 * 32]
    assert np.array_equal(cache.pool.cpu().numpy(), new.reshape(p.pool.shape))
    if scores:
        assert np.array_equal(cache.scores.cpu().numpy(), want)


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("W,heads,dim,page,per,first,keys", [(4, 4, 128, 64, 40, 700, 2500), (8, 2, 64, 32, 130, 0, 4160)])
def test_kv4_reorder_over_many_pages(cuda_ok, paged, W, heads, dim, page, per, first, keys):
    n, blocks, size = 2, page // 32, 32 * (dim + dim // 8)
    pages = n * W * per
    g = torch.Generator("cuda").manual_seed(W)
    pool = torch.randint(0, 256, (pages, heads * blocks * size), dtype=torch.uint8, device="cuda", generator=g)
    table = (torch.randperm(pages, device="cuda", generator=g) if paged else torch.arange(pages, device="cuda")).view(n * W, per)
    scores = torch.randn(n * W, heads, per * page, device="cuda", generator=g)
    cache = binding.Kv4Cache(pool.clone(), torch.full((n * W,), keys, dtype=torch.int32, device="cuda"), heads, dim, page,
                             table.int() if paged else None, scores.clone())
    par = torch.randint(0, W, (n, W), device="cuda", generator=g).int()
    binding.kv4_reorder(cache, par, first, keys)
    rows = (par.long() + torch.arange(n, device="cuda").unsqueeze(1) * W).flatten()

    def by_slot(x):   # [n * W][logical block][heads][bytes]
        return x.view(pages, heads, blocks, size)[table].transpose(2, 3).flatten(1, 2)
    b0, b1 = first // 32, -(-keys // 32)
    old, got = by_slot(pool), by_slot(cache.pool)
    want = old.clone()
    want[:, b0:b1] = old[rows][:, b0:b1]
    assert torch.equal(got, want)
    want = scores.clone()
    want[:, :, b0 * 32:b1 * 32] = scores[rows][:, :, b0 * 32:b1 * 32]
    assert torch.equal(cache.scores, want)


# ------------------------------------------------------------- the decoder

def _decoder(model, w, max_seq, batch, page):
    return binding.Decoder(model, w, max_seq, max_batch=batch, kv_page_tokens=page)


@pytest.mark.parametrize("page", [0, 64])
def test_kv_reorder_moves_the_decoders_cache(cuda_ok, page):
    model = synth.TINY
    w = {k: v.cuda() for k, v in synth.make_model(model, 0).items()}
    dec = _decoder(model, w, 160, 4, page)
    lens = [150, 130, 97, 20]
    toks = synth.make_prompt(sum(lens), model.vocab).cuda()
    dec.prefill_slots(toks, np.cumsum([0] + lens).tolist(), [2, 0, 3, 1])

    def caches(n):
        out = torch.zeros(4, model.n_layers, model.n_kv_heads, 2, n, model.head_dim, dtype=torch.bfloat16, device="cuda")
        for s in range(4):
            for l in range(model.n_layers):
                for h in range(model.n_kv_heads):
                    for i in range(2):
                        dec.copy_kv(s, l, h, i, n, out[s, l, h, i])
        torch.cuda.synchronize()
        return out
    if page:                                         # every slot has the pages that are compared
        dec.kv_reorder(torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda"), 0, 160)
    old = caches(160)
    slots = [3, 1, 2]
    dec.kv_reorder(torch.tensor([2, 0, 0], dtype=torch.int32, device="cuda"), 70, 150, slots)
    new = caches(160)
    want = old.clone()
    want[3, :, :, :, 70:150] = old[2, :, :, :, 70:150]
    want[1, :, :, :, 70:150] = old[3, :, :, :, 70:150]
    want[2, :, :, :, 70:150] = old[3, :, :, :, 70:150]
    assert torch.equal(new.view(torch.int16), want.view(torch.int16))
    for bad, code in ((dict(first=-1, n_pos=3), -5), (dict(first=4, n_pos=3), -5), (dict(first=0, n_pos=161), -5),
                      (dict(first=0, n_pos=3, slots=[0, 0, 1]), -1), (dict(first=0, n_pos=3, slots=[0, 4, 1]), -1)):
        with pytest.raises(binding.MkError) as e:
            dec.kv_reorder(torch.zeros(3, dtype=torch.int32, device="cuda"), **bad)
        assert e.value.code == code
    dec.close()


def test_kv_reorder_without_free_pages_is_refused(cuda_ok):
    model = synth.TINY
    w = {k: v.cuda() for k, v in synth.make_model(model, 0).items()}
    dec = binding.Decoder(model, w, 128, max_batch=2, kv_page_tokens=64, kv_pool_pages=3)
    dec.prefill_slots(synth.make_prompt(100, model.vocab).cuda(), [0, 100], [0])
    with pytest.raises(binding.MkError) as e:
        dec.kv_reorder(torch.zeros(2, dtype=torch.int32, device="cuda"), 0, 100)
    assert e.value.code == -2
    dec.kv_reorder(torch.zeros(2, dtype=torch.int32, device="cuda"), 0, 64)   # one page was left
    assert dec.status() == 0
    dec.close()


@pytest.mark.parametrize("page,beams,eos", [(0, 4, -1), (64, 3, -1), (0, 4, "seen"), (0, 1, -1)])
def test_beam_search_matches_a_search_by_prefills(cuda_ok, page, beams, eos):
    """The search on reordered caches against one on the host that prefills
    every hypothesis from its tokens: the same sequences and sums.  Cached and
    prefilled logits may differ by 3e-2 each (the library's own bar), a sum of
    5 steps of two of them by 0.3; where the host's hypotheses at the cut are
    closer than that, only the sums are compared."""
    model, n, steps = synth.TINY, 12, 5
    w = {k: v.cuda() for k, v in synth.make_model(model, 3).items()}
    # weights of this size give almost flat logits: an LM head 20 times larger tells tokens apart
    w["lm_head"] = (w["lm_head"].float() * 20).to(torch.bfloat16)
    prompt = synth.make_prompt(n, model.vocab).cuda()
    dec = _decoder(model, w, 64, max(beams, 2), page)
    if eos == "seen":
        eos = int(dec.beam_search(prompt, beams, 2)[0][1, 0])
    got, sums = dec.beam_search(prompt, beams, steps, eos=eos)
    torch.cuda.synchronize()
    assert dec.status() == 0
    host = _decoder(model, w, 64, 1, 0)
    logits = torch.empty(model.vocab, device="cuda")

    def log_probs(tokens):
        seq = torch.cat([prompt.cpu().int(), torch.tensor(tokens, dtype=torch.int32)]).cuda()
        host.prefill(seq, [0, len(seq)], logits)
        torch.cuda.synchronize()
        return torch.log_softmax(logits.double().cpu(), -1).numpy()

    hyps, close = [((), 0.0)], np.inf
    for _ in range(steps):
        found = []
        for toks, s in hyps:
            if eos >= 0 and eos in toks:
                found.append((toks + (eos,), s))
                continue
            lp = log_probs(list(toks))
            found += [(toks + (int(v),), s + lp[v]) for v in np.argsort(-lp)[:beams + 1]]
        found.sort(key=lambda f: -f[1])
        if len(found) > beams:
            close = min(close, found[beams - 1][1] - found[beams][1])
        hyps = found[:beams]
    sums = sums.cpu().numpy()
    assert (np.diff(sums) <= 0).all()
    bar = 0.3 * 20
    assert np.abs(sums - np.array([h[1] for h in hyps])).max() <= bar
    # each sequence's own sum, step by step, against prefills of its prefixes
    for row, s in zip(got.cpu().tolist(), sums):
        own, ended = 0.0, False
        for i, tok in enumerate(row):
            if not ended:
                own += log_probs(row[:i])[tok]
            else:
                assert tok == eos
            ended = ended or tok == eos
        assert abs(own - s) <= 0.05, (own, s)
    if close > 0.05:
        assert [tuple(r) for r in got.cpu().tolist()] == [h[0] for h in hyps]
    dec.close()
    host.close()


def test_beam_search_waits_for_its_prompt_and_is_waited_for(cuda_ok):
    """A decoder on a stream of its own, the prompt still being written on the
    caller's, the results read there at once: no wait on the host."""
    model = synth.TINY
    w = {k: v.cuda() for k, v in synth.make_model(model, 3).items()}
    prompt = synth.make_prompt(12, model.vocab).cuda()
    torch.cuda.synchronize()
    dec = binding.Decoder(model, w, 64, max_batch=4, stream=torch.cuda.Stream())
    first = dec.beam_search(prompt, 4, 8)
    torch.cuda.synchronize()
    want = [t.clone() for t in first]
    late = torch.zeros_like(prompt)
    torch.cuda.synchronize()
    for _ in range(3):
        late.zero_()
        torch.cuda._sleep(100_000_000)      # some 50 ms of the caller's stream
        late.copy_(prompt)
        got = dec.beam_search(late, 4, 8)
        seen = [t.clone() for t in got]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(seen, want))
    assert dec.status() == 0
    dec.close()


@pytest.mark.parametrize("mseed,pseed,beams,page,eos", [
    (3, 3, 3, 0, False), (3, 3, 4, 64, False), (4, 1, 4, 0, False), (3, 4, 3, 64, False), (5, 2, 4, 0, False),
    (3, 5, 3, 0, True), (4, 2, 3, 64, True), (3, 2, 4, 0, True)])
def test_beam_search_matches_a_search_that_replays_every_hypothesis(cuda_ok, mseed, pseed, beams, page, eos):
    """Against a search on the host whose hypotheses are decoded from the prompt
    again at every step, each in the slot where the search holds it: the same
    kernels on the same tokens, so the logits are the same and only the
    selection's sums differ, 2^-18 and a rounding to fp32 a step.  The prompts
    are such that all choices lie further apart; then tokens, order and sums follow."""
    model, n, steps = synth.TINY, 12, 6
    w = {k: v.cuda() for k, v in synth.make_model(model, mseed).items()}
    w["lm_head"] = (w["lm_head"].float() * 20).to(torch.bfloat16)      # logits that tell tokens apart
    prompt = synth.make_prompt(n, model.vocab, pseed).cuda()
    dec, host = (_decoder(model, w, 64, beams, page) for _ in range(2))
    end = int(dec.beam_search(prompt, beams, 2)[0][1, 0]) if eos else -1
    got, sums = dec.beam_search(prompt, beams, steps, eos=end)
    logits = torch.empty(beams, model.vocab, device="cuda")
    slots = list(range(beams))
    hyps, close = [((), 0.0)], np.inf
    for s in range(steps):
        for b in slots:
            host.prefill_slots(prompt, [0, n], [b], logits[b:b + 1])
        for i in range(s):
            toks = torch.tensor([h[0][i] for h in hyps], dtype=torch.int32, device="cuda")
            host.decode_slots(toks, [n + i] * beams, slots, logits)
        lp = torch.log_softmax(logits.double(), -1).cpu().numpy()
        found = []
        for b, (toks, total) in enumerate(hyps):
            if end in toks:
                found.append((toks + (end,), total))
            else:
                found += [(toks + (int(v),), total + lp[b, v]) for v in np.argsort(-lp[b], kind="stable")[:beams + 1]]
        found.sort(key=lambda f: -f[1])
        close = min([close] + [a[1] - b[1] for a, b in zip(found[:beams], found[1:])])
        hyps = found[:beams]
    torch.cuda.synchronize()
    bar = steps * (2.0 ** -18 + 2.0 ** -24 * abs(hyps[-1][1]))
    assert close > 2 * bar, close
    assert [tuple(r) for r in got.cpu().tolist()] == [h[0] for h in hyps]
    assert np.abs(sums.cpu().numpy() - np.array([h[1] for h in hyps])).max() <= bar
    assert not eos or any(end in h[0] for h in hyps)
    assert dec.status() == 0 and host.status() == 0
    dec.close()
    host.close()


def test_beam_search_refuses_other_prompts(cuda_ok):
    """Token ids of another type, on the host or with gaps: read as int32 they
    would be another prompt."""
    model = synth.TINY
    w = {k: v.cuda() for k, v in synth.make_model(model, 3).items()}
    dec = _decoder(model, w, 64, 2, 0)
    prompt = synth.make_prompt(12, model.vocab)
    for bad in (prompt.cuda().long(), prompt, prompt.cuda().repeat_interleave(2)[::2]):
        with pytest.raises(TypeError):
            dec.beam_search(bad, 2, 3)
    for beams, steps in ((0, 3), (3, 3), (2, 0), (2, 54)):
        with pytest.raises(ValueError):
            dec.beam_search(prompt.cuda(), beams, steps)
    assert dec.status() == 0
    dec.close()
