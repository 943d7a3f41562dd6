"""The 4-bit KV cache on the GPU: append, read, attention and eviction against
the plain reference in 64 bits, at the sizes, masks and contents where they
can go wrong, and all of them together as a decode uses them.

Codes, scales, kept slots and moved bytes are compared exactly.  Attention is
held to a bound from its arithmetic (see _bound)."""
import numpy as np
import pytest
import torch

from persistent_megakernel_03_b200 import binding
from kv4_util import GROUP, TINY, Plain, attend, values

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
# rounding of a probability that enters the product: one fp16 part, or two
PART = {torch.float32: 2.0 ** -22, torch.float16: 2.0 ** -22, torch.bfloat16: 2.0 ** -12}


def _bound(out, mass, reach, dtype):
    """Largest error of an output element.

    A score is a sum of products of 22-bit queries and exact keys, added in
    fp32 over at most 8 steps of 16 for each of 2 parts, an addition of the
    tensor core losing up to 2^-22 of the running size: 2^-18 of scale *
    sum |q||k| covers it, and the same again the scaling to log2 units.  A
    weight is then off by the exponential of that (numerator and sum: twice),
    by its part, and by fp32 sums (2^-18 for up to 64 partial sums in a row);
    the result is rounded once -- to half a step of its size, and below the
    type's normal range to half the smallest step there (fp16: 2^-25)."""
    s = 2 * 2.0 ** -18 * reach[..., None]
    f = torch.finfo(dtype)
    return np.abs(out) * f.eps / 2 + mass * (2 * s + PART[dtype] + 2.0 ** -18) + f.tiny * f.eps / 2


def _cuda(p, lens, scores=None):
    return binding.Kv4Cache(torch.from_numpy(p.pool.copy()).cuda(),
                            torch.tensor(lens, dtype=torch.int32, device="cuda"), p.heads, p.dim, p.page,
                            torch.from_numpy(p.table.copy()).cuda(),
                            None if scores is None else torch.from_numpy(scores.astype(np.float32)).cuda(),
                            *p.log2)


def _workspace(c, q_len, heads, acc):
    n = binding.attention_kv4_workspace_bytes(c, q_len, heads, acc)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN, if read before written


def _attend(c, q, acc=False, scale=None, out=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if out is None else out
    binding.attention_kv4(c, q, out, _workspace(c, q.shape[1], q.shape[2], acc), scale, acc)
    return out


def _check(p, lens, q, out, scale, scores=None, before=None, skip=()):
    T, Hq = q.shape[1], q.shape[2]
    qd, od = q.double().cpu().numpy(), out.double().cpu().numpy()
    for s, n in enumerate(lens):
        if s in skip:
            continue
        n = min(max(n, 0), p.capacity)
        k, v = p.read(s, n)
        want, w, mass, reach = attend(qd[s], k, v, scale, Hq // p.heads)
        err = np.abs(od[s] - want)
        tol = _bound(want, mass, reach, q.dtype)
        assert np.array_equal(np.isnan(od[s]), np.isnan(want)), f"sequence {s}: NaN in other places"
        ok = ~np.isnan(want)
        assert (err[ok] <= tol[ok]).all(), f"sequence {s}: {np.nanmax(err / tol)} times the bound"
        if scores is not None:
            got = scores[s, :, :n].double().cpu().numpy() - before[s, :, :n]
            # a weight as above, then added to what was there in fp32
            t = 4 * 2.0 ** -18 * (reach.max() if reach.size else 0) + 2.0 ** -17
            lim = w * t + (np.abs(before[s, :, :n]) + w) * 2.0 ** -23 * 2 + 1e-30
            assert (np.abs(got - w) <= lim).all(), f"sequence {s}: scores"
            assert np.array_equal(scores[s, :, n:].cpu().numpy(), before[s, :, n:].astype(np.float32))


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,dim,page,counts,old", [
    (1, 64, 32, [1], [0]), (2, 64, 64, [1, 1, 1], [31, 32, 63]), (8, 128, 64, [5, 0, 70], [3, 9, 0]),
    (3, 128, 96, [100, 1], [0, 95]), (2, 64, 32, [0, 0, 33, 0], [1, 2, 3, 4]),
    (33, 64, 32, [3, 2], [0, 31]), (40, 128, 32, [1, 3], [5, 0]), (1, 64, 32, [1] * 600, [i % 7 for i in range(600)]),
])
def test_append_writes_the_format(cuda_ok, dtype, heads, dim, page, counts, old):
    lens = [a + b for a, b in zip(old, counts)]
    p = Plain(len(lens), heads, dim, page, -(-max(max(lens), 1) // page), seed=3, fill=0xA5, k_log2=1, v_log2=-2)
    rng = np.random.default_rng(dim + len(lens))
    n = sum(counts)
    kv = []
    for w in (0, 1):
        x = rng.normal(size=(n, heads, dim)) * np.exp(rng.normal(size=(1, heads, dim)))
        x[rng.random(x.shape) < 0.05] = 0.0
        x.reshape(-1)[::7] = rng.choice([0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -6.0, 0.25], x.reshape(-1)[::7].shape)
        kv.append(torch.from_numpy(x).to(TYPES[dtype]))
    scores = np.full((len(lens), heads, p.capacity), 3.5)
    c = _cuda(p, lens, scores)
    offs = np.cumsum([0] + counts)
    # tokens of a fused row: strides above heads * dim
    wide = torch.zeros(n, 2 * heads + 1, dim, dtype=TYPES[dtype])
    wide[:, :heads], wide[:, heads:2 * heads] = kv
    wide = wide.cuda()
    binding.kv4_append(c, wide[:, :heads], wide[:, heads:2 * heads],
                       torch.from_numpy(offs.astype(np.int32)).cuda())
    for s, m in enumerate(counts):
        for j in range(m):
            p.write(s, old[s] + j, kv[0][offs[s] + j].double().numpy(), kv[1][offs[s] + j].double().numpy())
            scores[s, :, old[s] + j] = 0.0
    assert np.array_equal(c.pool.cpu().numpy(), p.pool)
    assert np.array_equal(c.scores.cpu().numpy(), scores.astype(np.float32))


def test_append_rounds_borders_exactly(cuda_ok):
    """Group maxima on, just above and just below 6 times every midpoint of the
    scales, and elements the same about every midpoint of the codes."""
    from kv4_util import E4M3
    mids = np.float32(6 * (E4M3[1:] + E4M3[:-1]) / 2)
    tops = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(1e9)),
                           np.float32(6 * E4M3), np.float32([2688, 2700, 1e30, 3.4e38, 1e-30, 0.0])]).astype(np.float32)
    n = len(tops)
    x = np.zeros((n, 1, 64), np.float32)
    cm = np.float32([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    from kv4_util import quantize
    for i, t in enumerate(tops):
        for g in range(4):
            x[i, 0, 16 * g] = t if g % 2 else -t
            s = E4M3[min(quantize(x[i, 0, 16 * g:16 * g + 16])[1][0], 126)]
            b = np.float32(cm * np.float32(s))
            x[i, 0, 16 * g + 1:16 * g + 8] = [b, np.nextafter(b, np.float32(0)), np.nextafter(b, np.float32(1e9)), -b][g]
            big = np.abs(x[i, 0, 16 * g + 1:16 * g + 8]) > abs(t)
            x[i, 0, 16 * g + 1:16 * g + 8][big] = 0
    p = Plain(1, 1, 64, 32, -(-n // 32), seed=1)
    c = _cuda(p, [n])
    t = torch.from_numpy(x).cuda()
    binding.kv4_append(c, t, t, torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    for j in range(n):
        p.write(0, j, x[j], x[j])
    assert np.array_equal(c.pool.cpu().numpy(), p.pool)


def test_append_nan_and_infinity_make_their_group_nan(cuda_ok):
    x = torch.ones(3, 2, 64)
    x[0, 0, 5], x[1, 1, 20], x[2, 0, 63] = float("nan"), float("inf"), float("-inf")
    p = Plain(1, 2, 64, 32, 1)
    c = _cuda(p, [3])
    binding.kv4_append(c, x.cuda(), x.cuda(), torch.tensor([0, 3], dtype=torch.int32, device="cuda"))
    k = torch.zeros(1, 3, 2, 64, device="cuda")
    v = torch.zeros_like(k)
    binding.kv4_read(c, k, v)
    want = torch.isfinite(x.view(3, 2, 4, 16)).all(-1, keepdim=True).expand(3, 2, 4, 16).reshape(3, 2, 64)
    for y in (k, v):
        assert torch.equal(torch.isfinite(y[0]).cpu(), want)
        # ones: 1/6 lies between the scales 10/64 and 11/64, nearer the second; 6 * 11/64
        assert torch.equal(y[0].cpu()[want], torch.full((int(want.sum()),), 1.03125))


def test_append_skips_what_has_no_place(cuda_ok):
    """Lengths below the count and above the capacity, bad pages, tokens
    outside the offsets: nothing else changes."""
    p = Plain(3, 1, 64, 32, 2, seed=5, n_pages=8, fill=0x33)
    p.table[1, 0] = -1
    p.table[2, 1] = 99
    lens = [66, 34, 33]
    c = _cuda(p, lens)
    x = torch.randn(14, 1, 64)
    offs = [1, 5, 9, 12]          # token 0 and tokens 12, 13 belong to nobody
    binding.kv4_append(c, x.cuda(), x.cuda(), torch.tensor(offs, dtype=torch.int32, device="cuda"))
    for s in range(3):
        for j in range(offs[s], offs[s + 1]):
            slot = lens[s] - offs[s + 1] + j
            if 0 <= slot < p.capacity and 0 <= p.table[s, slot // 32] < 8:
                p.write(s, slot, x[j].double().numpy(), x[j].double().numpy())
    assert np.array_equal(c.pool.cpu().numpy(), p.pool)


# -------------------------------------------------------------------- read

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,page", [(64, 32), (128, 96)])
def test_read_gives_the_values_and_leaves_the_rest(cuda_ok, dtype, dim, page):
    lens = [0, 1, 33, 95, 200]
    p = Plain(5, 3, dim, page, -(-100 // page), seed=9, k_log2=-3, v_log2=2)
    p.fill_random([100] * 5)
    p.table[3, 0] = -7
    c = _cuda(p, lens)
    n = 97
    k = torch.full((5, n, 3, dim), 9.0, dtype=TYPES[dtype], device="cuda")
    v = torch.full_like(k, 8.0)
    binding.kv4_read(c, k, v)
    for s, m in enumerate(lens):
        m = min(m, p.capacity, n)
        lo = page if s == 3 else 0
        p.table[3, 0] = 0
        a, b = p.read(s, m)
        for x, y, fill in ((k, a, 9.0), (v, b, 8.0)):
            x = x[s].double().cpu().numpy()
            assert np.array_equal(x[lo:m], y[lo:])      # <= 6 significant bits: exact in every type
            assert (x[m:] == fill).all() and (x[:min(lo, m)] == fill).all()


# --------------------------------------------------------------- attention

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,heads,group,dim,q_len,page,acc", [
    ([1], 1, 1, 64, 1, 32, True), ([1], 2, 8, 128, 1, 32, False), ([32], 1, 4, 128, 1, 32, True),
    ([33, 31, 0], 2, 7, 64, 1, 64, True), ([551], 2, 7, 64, 1, 576, False),
    ([700, 65, 1, 2049], 8, 4, 128, 1, 64, True), ([5], 1, 16, 128, 1, 32, True),
    ([3, 0, 40, 129], 2, 4, 128, 5, 32, True), ([40, 7], 1, 9, 64, 3, 64, True),
    ([64, 96], 3, 5, 64, 8, 96, True), ([2], 1, 8, 128, 16, 32, True), ([300], 1, 1, 64, 33, 64, True),
    ([257] * 40, 1, 2, 64, 1, 32, True), ([0, 0], 2, 2, 64, 2, 32, True), ([90, 3], 2, 4, 128, 10, 32, True),
    ([i % 5 * 9 for i in range(700)], 1, 1, 64, 1, 64, True), ([100, 33], 1, 8, 128, 3, 64, False),
])
def test_attention_matches_the_reference(cuda_ok, dtype, lens, heads, group, dim, q_len, page, acc):
    p = Plain(len(lens), heads, dim, page, -(-max(max(lens), 1) // page), seed=len(lens), k_log2=1, v_log2=-1)
    p.fill_random(lens, size=1.5)
    g = torch.Generator().manual_seed(dim + q_len)
    q = torch.randn(len(lens), q_len, heads * group, dim, generator=g).to(TYPES[dtype]).cuda()
    before = np.abs(np.random.default_rng(2).normal(size=(len(lens), heads, p.capacity))).astype(np.float32)
    c = _cuda(p, lens, before)
    out = _attend(c, q, acc)
    _check(p, lens, q, out, dim ** -0.5, c.scores if acc else None, before.astype(np.float64))
    if not acc:
        assert np.array_equal(c.scores.cpu().numpy(), before)


def test_attention_long_context(cuda_ok):
    lens = [20011, 32768]
    p = Plain(2, 2, 128, 64, 512, seed=1)
    p.fill_random(lens, size=1.0)
    q = torch.randn(2, 1, 8, 128, generator=torch.Generator().manual_seed(0)).cuda()
    before = np.zeros((2, 2, p.capacity))
    c = _cuda(p, lens, before)
    out = _attend(c, q, True)
    # values by whole arrays: the reference's reader is slow here
    k = torch.zeros(2, 32768, 2, 128, device="cuda")
    v = torch.zeros_like(k)
    binding.kv4_read(c, k, v)
    assert np.array_equal(k[0, 777:780].double().cpu().numpy(), p.read(0, 780)[0][777:])
    for s, n in enumerate(lens):
        kd, vd = (x[s, :n].double().cpu().numpy() for x in (k, v))
        want, w, mass, reach = attend(q[s].double().cpu().numpy(), kd, vd, 128 ** -0.5, 4)
        tol = _bound(want, mass, reach, q.dtype)
        assert (np.abs(out[s].double().cpu().numpy() - want) <= tol).all()
        t = 4 * 2.0 ** -18 * reach.max() + 2.0 ** -17
        assert (np.abs(c.scores[s, :, :n].double().cpu().numpy() - w) <= w * t + 1e-30).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_with_queries_of_all_sizes(cuda_ok, dtype, dim):
    """Rows from 2^-100 (fp16: 2^-14) to 2^14, a zero row and a spike: the
    power-of-two scaling of a row loses nothing."""
    p = Plain(1, 1, dim, 32, 4, seed=2)
    p.fill_random([100], size=1.0)
    lo = -14 if dtype == "fp16" else -100
    g = torch.Generator().manual_seed(4)
    q = torch.randn(1, 1, 8, dim, generator=g) * 2.0 ** torch.tensor([lo, -8, 0, 2, 3, 4, 14, 0.0]).view(1, 1, 8, 1)
    q[0, 0, 7] = 0
    q[0, 0, 2, 3] = 60.0
    q = q.to(TYPES[dtype]).cuda()
    c = _cuda(p, [100])
    out = _attend(c, q)
    _check(p, [100], q, out, dim ** -0.5)
    out = _attend(c, q, scale=0.001)
    _check(p, [100], q, out, float(np.float32(0.001)))


@pytest.mark.parametrize("q_len", [1, 4])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_ignores_what_is_masked(cuda_ok, dim, q_len):
    """NaN scales behind the last key, in pages that are nobody's, and in a
    whole block that a bad page would give; lengths out of range."""
    lens = [37, 70, 4000, -3, 64]
    p = Plain(5, 2, dim, 32, 3, seed=3, n_pages=20)
    p.fill_random([96] * 5)
    p.table[4, 1] = 77                               # slots 32..63 of sequence 4 have no page
    clean = p.pool.copy()
    half = 32 * (dim // 2 + dim // GROUP)
    blocks = p.pool.reshape(20, 2, 1, 2, half)
    used = set(p.table.reshape(-1).tolist())
    for page in range(20):
        if page not in used:
            blocks[page, ..., 32 * dim // 2:] = 0x7F
    for s, n in enumerate(lens):
        for slot in range(min(max(n, 0), 96), 96):
            if p.table[s, slot // 32] < 20:
                sc = blocks[p.table[s, slot // 32], :, 0, :, 32 * dim // 2:].reshape(2, 2, 32, dim // GROUP)
                sc[:, :, slot % 32] = 0x7F
    q = torch.randn(5, q_len, 4, dim, generator=torch.Generator().manual_seed(1)).cuda()
    before = np.zeros((5, 2, 96))
    c = _cuda(p, lens, before)
    out = _attend(c, q, True)
    assert torch.isfinite(out).all() and torch.isfinite(c.scores).all()
    _check(p, lens, q, out, dim ** -0.5, c.scores, before, skip=(4,))
    # sequence 4 sees slots 0..31 only, its tokens all of them
    k, v = Plain.read(p, 4, 32)
    qd = q[4].double().cpu().numpy()
    for i in range(q_len):
        want, w, mass, reach = attend(qd[i:i + 1], k, v, dim ** -0.5, 2)
        assert (np.abs(out[4, i:i + 1].double().cpu().numpy() - want) <= _bound(want, mass, reach, q.dtype)).all()
    assert (c.scores[4, :, 32:] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,group", [(64, 1), (128, 3)])
def test_attention_nan_reaches_only_rows_that_see_it(cuda_ok, dim, group, dtype):
    """A NaN group in the value of the second newest key: earlier tokens do not
    see it.  A NaN key makes the rows that see it NaN."""
    lens, q_len = [45, 45], 4
    p = Plain(2, 1, dim, 32, 2, seed=8)
    p.fill_random(lens)
    for s, w in ((0, 1), (1, 0)):
        page, at = p._at(s, 43, 0)
        p.pool[page, at[w][1] + 1] = 0x7F      # dims 16..31
    q = torch.randn(2, q_len, group, dim, generator=torch.Generator().manual_seed(6)).to(TYPES[dtype]).cuda()
    c = _cuda(p, lens)
    out = _attend(c, q)
    nan = torch.isnan(out).cpu()
    assert not nan[:, :2].any()
    assert nan[1, 2:].all()
    want = torch.zeros(group, dim, dtype=torch.bool)
    want[:, 16:32] = True
    assert torch.equal(nan[0, 2], want) and torch.equal(nan[0, 3], want)
    k, v = p.read(0, 45)
    o, w, mass, reach = attend(q[0].double().cpu().numpy(), k, np.nan_to_num(v), dim ** -0.5, group)
    ok = ~nan[0].numpy()
    assert (np.abs(out[0].double().cpu().numpy() - o)[ok] <= _bound(o, mass, reach, q.dtype)[ok]).all()


def _with_bad_row(cuda_ok, dtype, dim, group, n, bad):
    """Token 1 of 4 has one query head with a bad element: (plain cache, clean
    queries, cache with scores, outputs)."""
    p = Plain(1, 2, dim, 32, -(-n // 32), seed=7)
    p.fill_random([n])
    q = torch.randn(1, 4, 2 * group, dim, generator=torch.Generator().manual_seed(6)).to(TYPES[dtype])
    q[0, 1, 0] = 0
    dirty = q.clone()
    dirty[0, 1, 0, 5] = bad
    c = _cuda(p, [n], np.zeros((1, 2, p.capacity)))
    return p, q, c, _attend(c, dirty.cuda(), True)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,group,n", [(64, 1, 45), (128, 4, 2003), (64, 9, 300)])
def test_attention_bad_query_row_stays_alone(cuda_ok, dim, group, n, dtype, bad):
    """A NaN or an infinity in one query row: that row is NaN and so are the
    scores of the keys that it sees; other rows, and the keys that only later
    tokens see, are as without it."""
    p, q, c, out = _with_bad_row(cuda_ok, dtype, dim, group, n, bad)
    nan = torch.isnan(out[0]).cpu()
    assert nan[1, 0].all() and int(nan.sum()) == dim
    k, v = p.read(0, n)
    want, w, mass, reach = attend(q[0].double().numpy(), k, v, dim ** -0.5, group)
    ok = ~nan.numpy()
    assert (np.abs(out[0].double().cpu().numpy() - want)[ok] <= _bound(want, mass, reach, q.dtype)[ok]).all()
    got = c.scores[0, :, :n].double().cpu().numpy()
    assert np.isnan(got[0, :n - 2]).all()
    t = 4 * 2.0 ** -18 * reach.max() + 2.0 ** -17
    for a, b in ((got[0, n - 2:], w[0, n - 2:]), (got[1], w[1])):
        assert (np.abs(a - b) <= b * t + b * 2.0 ** -22 + 1e-30).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,n", [(64, 3), (128, 700)])
def test_attention_row_of_minus_infinities_is_not_an_empty_one(cuda_ok, dim, n, dtype):
    """An infinite query against keys of one sign: every score is -inf, and the
    softmax of that is NaN, not the zeros of a row that sees nothing."""
    k = -torch.ones(n, 1, dim)
    p = Plain(1, 1, dim, 32, -(-n // 32), seed=1)
    c = _cuda(p, [n])
    binding.kv4_append(c, k.cuda(), torch.ones(n, 1, dim).cuda(), torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    q = torch.zeros(1, 1, 2, dim)
    q[0, 0, 1] = float("inf")
    out = _attend(c, q.to(TYPES[dtype]).cuda())
    assert torch.isnan(out[0, 0, 1]).all()
    # 1/6 is nearest 11/64: ones read back as 6 * 11/64; a mean of equal values
    want = torch.full((dim,), 1.03125)
    assert ((out[0, 0, 0].float().cpu() - want).abs() <= 1.03125 * (torch.finfo(TYPES[dtype]).eps / 2 + PART[TYPES[dtype]] + 2.0 ** -18)).all()


@pytest.mark.parametrize("dtype,scale,k_log2", [
    ("fp32", 1.0, 0), ("bf16", 1.0, 0), ("fp32", 2.0 ** 59, 32), ("bf16", 2.0 ** 59, 32), ("fp16", 2.0 ** 59, 32),
    ("fp32", 2.0 ** -59, 0)])
@pytest.mark.parametrize("dim,n", [(64, 40), (128, 1500)])
def test_attention_of_scores_past_fp32(cuda_ok, dim, n, dtype, scale, k_log2):
    """Finite queries whose scores pass fp32's range: the highest key takes all
    the weight (equal ones share it).  Queries and keys are powers of two times
    few bits, so their products and sums are exact here: no error of the scores
    enters the bound."""
    p = Plain(1, 2, dim, 32, -(-n // 32), seed=3, k_log2=k_log2)
    p.fill_random([n], size=1.0)
    g = torch.Generator().manual_seed(dim)
    top = 15 if dtype == "fp16" else 127
    q = torch.where(torch.rand(1, 2, 6, dim, generator=g) < 0.5, 1.0, -1.0) * 2.0 ** (
        top - torch.randint(0, 3, (1, 2, 6, dim), generator=g).float())
    q = q.to(TYPES[dtype]).cuda()
    assert torch.isfinite(q).all()
    c = _cuda(p, [n], np.zeros((1, 2, p.capacity)))
    out = _attend(c, q, True, scale)
    k, v = p.read(0, n)
    want, w, mass, _ = attend(q[0].double().cpu().numpy(), k, v, scale, 3)
    tol = np.abs(want) * torch.finfo(q.dtype).eps / 2 + mass * (PART[q.dtype] + 2.0 ** -18) + 2.0 ** -25
    assert (np.abs(out[0].double().cpu().numpy() - want) <= tol).all()
    assert (np.abs(c.scores[0, :, :n].double().cpu().numpy() - w) <= w * 2.0 ** -17 + 1e-30).all()


def _reference64(c, q, scale):
    """out, weights, and the bound's sums of attention over a cache's values as
    read back, in 64 bits on the GPU, one sequence after another."""
    n_seq, T, Hq, d = q.shape
    group = Hq // c.n_kv_heads
    n = int(c.lens.max())
    k = torch.zeros(n_seq, n, c.n_kv_heads, d, device="cuda")
    v = torch.zeros_like(k)
    binding.kv4_read(c, k, v)
    for s in range(n_seq):
        m = int(c.lens[s])
        kd = k[s, :m].double().transpose(0, 1).repeat_interleave(group, 0)          # [Hq][m][d]
        vd = v[s, :m].double().transpose(0, 1).repeat_interleave(group, 0)
        qd = q[s].double().transpose(0, 1)                                          # [Hq][T][d]
        seen = torch.arange(m, device="cuda") < (m - T + 1 + torch.arange(T, device="cuda")).unsqueeze(-1)
        x = (qd @ kd.transpose(1, 2) * scale).masked_fill(~seen, -float("inf"))
        p = torch.softmax(x, -1).nan_to_num(0.0)
        small = TINY * p.amax(-1, keepdim=True) * seen
        reach = (qd.abs() @ kd.abs().transpose(1, 2) * scale).masked_fill(~seen, 0.0).amax(-1)
        yield (s, m, (p @ vd).transpose(0, 1).cpu().numpy(), p.unflatten(0, (-1, group)).sum((1, 2)).cpu().numpy(),
               ((p + small) @ vd.abs()).transpose(0, 1).cpu().numpy(), reach.transpose(0, 1).cpu().numpy())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n_seq,lo,hi,heads,group,dim,q_len,page", [
    (12, 6001, 8191, 8, 4, 128, 1, 128), (24, 3000, 4097, 4, 8, 64, 1, 64),    # long batches
    (3, 500, 2100, 2, 8, 128, 6, 64), (2, 900, 1301, 4, 8, 128, 16, 32),       # 48 and 128 rows of a KV head
    (2, 700, 2049, 1, 16, 128, 64, 64), (3, 1, 1500, 2, 5, 64, 33, 96),        # 1,024 rows; 165, with a short sequence
])
def test_attention_at_size(cuda_ok, dtype, n_seq, lo, hi, heads, group, dim, q_len, page):
    rng = np.random.default_rng(hi)
    lens = [lo, hi] + rng.integers(lo, hi + 1, n_seq - 2).tolist()
    p = Plain(n_seq, heads, dim, page, -(-hi // page), seed=n_seq, k_log2=-1, v_log2=2)
    p.fill_random(lens, size=1.5)
    q = torch.randn(n_seq, q_len, heads * group, dim, generator=torch.Generator().manual_seed(hi)).to(TYPES[dtype]).cuda()
    c = _cuda(p, lens, np.zeros((n_seq, heads, p.capacity)))
    out = _attend(c, q, True)
    for s, m, want, w, mass, reach in _reference64(c, q, dim ** -0.5):
        err, tol = np.abs(out[s].double().cpu().numpy() - want), _bound(want, mass, reach, q.dtype)
        assert (err <= tol).all(), (s, (err / tol).max())
        # a weight as in _check; up to 1,024 of them added one after another in fp32
        t = 4 * 2.0 ** -18 * reach.max() + 2.0 ** -17 + q_len * group * 2.0 ** -24
        got = c.scores[s].double().cpu().numpy()
        assert (np.abs(got[:, :m] - w) <= w * t + 1e-30).all(), s
        assert (got[:, m:] == 0).all()


def test_attention_small_weights_add_up(cuda_ok):
    """One key far above thousands of equal ones: each of their weights is 2^-20
    of the first, together they are not."""
    n, dim = 20000, 64
    p = Plain(1, 1, dim, 32, 625)
    blocks = p.pool.reshape(625, 1, 1, 2, -1)
    half = 32 * dim // 2
    blocks[..., half:] = 7 * 8                    # scales 1
    blocks[:, :, :, 1, :half] = 0x22              # values 1
    page, at = p._at(0, 4321, 0)
    p.pool[page, at[0][0]] = 0x07                 # key: 6 in dim 0
    p.pool[page, at[1][0]:at[1][0] + dim // 2] = 0xAA   # value: -1
    q = torch.zeros(1, 1, 1, dim)
    q[..., 0] = 20 * np.log(2) / 6 * 8            # score 20 ln 2 with scale 1/8
    for t in TYPES.values():
        qq = q.to(t).cuda()
        out = _attend(_cuda(p, [n]), qq)
        _check_whole = np.exp(qq.double().cpu().numpy()[0, 0, 0, 0] * 6 / 8)
        want = ((n - 1) - _check_whole) / ((n - 1) + _check_whole)
        tol = abs(want) * torch.finfo(t).eps / 2 + PART[t] + 2.0 ** -17 + 2 * 2.0 ** -17 * 14
        assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


def test_attention_strided_queries_and_one_page_without_table(cuda_ok):
    p = Plain(3, 2, 64, 96, 1, seed=0)
    p.table[:] = np.arange(3).reshape(3, 1)
    lens = [96, 5, 50]
    p.fill_random(lens)
    fused = torch.randn(3, 2, 4 + 2 + 2, 64, generator=torch.Generator().manual_seed(2)).cuda()
    q = fused[:, :, :4]
    c = _cuda(p, lens)
    bare = binding.Kv4Cache(c.pool, c.lens, 2, 64, 96)
    out = torch.empty(3, 2, 4, 64, device="cuda")
    binding.attention_kv4(bare, q, out, _workspace(bare, 2, 4, False))
    _check(p, lens, q, out, 0.125)
    assert torch.equal(out, _attend(c, q.contiguous()))


def test_addresses_that_are_only_16_byte_aligned(cuda_ok):
    """Rows 16 bytes off a 32-byte boundary, in and out."""
    for dtype in TYPES.values():
        off = 16 // torch.empty((), dtype=dtype).element_size()
        p = Plain(1, 2, 64, 32, 2, seed=1)
        c = _cuda(p, [50])
        raw = torch.randn(2, 50 * 128 + off, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
        k, v = (x[off:].view(50, 2, 64) for x in raw)
        assert k.data_ptr() % 32 == 16
        binding.kv4_append(c, k, v, torch.tensor([0, 50], dtype=torch.int32, device="cuda"))
        for j in range(50):
            p.write(0, j, k[j].double().cpu().numpy(), v[j].double().cpu().numpy())
        assert np.array_equal(c.pool.cpu().numpy(), p.pool)
        back = torch.zeros(2, 50 * 128 + off, dtype=dtype, device="cuda")
        ko, vo = (x[off:].view(1, 50, 2, 64) for x in back)
        binding.kv4_read(c, ko, vo)
        for x, y in zip((ko, vo), p.read(0, 50)):
            assert np.array_equal(x[0].double().cpu().numpy(), y)
        q = torch.randn(2 * 64 + off, generator=torch.Generator().manual_seed(2)).to(dtype).cuda()[off:].view(1, 1, 2, 64)
        out = torch.zeros(2 * 64 + off, dtype=dtype, device="cuda")[off:].view(1, 1, 2, 64)
        _check(p, [50], q, _attend(c, q, out=out), 0.125)


def test_pools_past_32_bits(cuda_ok):
    """Pages whose bytes lie 5 GB into the pool, through every operator."""
    heads, dim, page, pages = 8, 128, 64, 70000
    size = heads * page * (dim + dim // 8)
    pool = torch.zeros(pages, size, dtype=torch.uint8, device="cuda")
    table = torch.tensor([[pages - 1, 60000], [65000, 2]], dtype=torch.int32, device="cuda")
    lens = [100, 70]
    p = Plain(2, heads, dim, page, 2, seed=1)
    p.table = np.array([[0, 1], [2, 3]], np.int32)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2, 170, heads, dim, generator=g)
    for s, a in ((0, 0), (1, 100)):
        for j in range(lens[s]):
            p.write(s, j, x[0, a + j].double().numpy(), x[1, a + j].double().numpy())
    scores = torch.zeros(2, heads, 128, device="cuda")
    c = binding.Kv4Cache(pool, torch.tensor(lens, dtype=torch.int32, device="cuda"), heads, dim, page, table, scores)
    k, v = x.cuda()
    binding.kv4_append(c, k, v, torch.tensor([0, 100, 170], dtype=torch.int32, device="cuda"))
    assert np.array_equal(pool[table.view(-1).long()].cpu().numpy(), p.pool)
    q = torch.randn(2, 1, 32, dim, generator=g).cuda()
    out = _attend(c, q, True)
    _check(p, lens, q, out, dim ** -0.5, scores, np.zeros((2, heads, 128)))
    dst_table = torch.tensor([[69998], [69997]], dtype=torch.int32, device="cuda")
    dst = binding.Kv4Cache(pool, torch.tensor([64, 64], dtype=torch.int32, device="cuda"), heads, dim, page, dst_table,
                           torch.zeros(2, heads, 64, device="cuda"))
    kept = torch.zeros(2, heads, 64, dtype=torch.int32, device="cuda")
    before = scores.cpu().numpy()
    binding.kv4_evict(c, dst, 64, 4, 8, kept)
    ko = torch.zeros(2, 64, heads, dim, device="cuda")
    vo = torch.zeros_like(ko)
    binding.kv4_read(dst, ko, vo)
    for s in range(2):
        a, b = p.read(s, lens[s])
        for h in range(heads):
            want = _kept(before[s, h], lens[s], 64, 4, 8)
            assert kept[s, h].tolist() == want
            assert np.array_equal(ko[s, :, h].double().cpu().numpy(), a[want, h])
            assert np.array_equal(vo[s, :, h].double().cpu().numpy(), b[want, h])
    par = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    old = pool[dst_table.view(-1).long()].clone()
    binding.kv4_reorder(dst, par, 0, 64)
    assert torch.equal(pool[dst_table.view(-1).long()], old.flip(0))


def test_attention_over_millions_of_keys(cuda_ok):
    """One head's 2.6 million keys in small pages: a warp's range runs over more
    pages than it looks up at once.  Against 64 bits on the values read back."""
    n, dim, page = 2_600_001, 64, 32
    pages = -(-n // page)
    pool = torch.randint(0, 256, (pages, page * (dim + dim // 8)), dtype=torch.uint8, device="cuda",
                         generator=torch.Generator("cuda").manual_seed(1))
    half = page * (dim // 2 + dim // 16)
    blocks = pool.view(pages, 2, half)
    blocks[:, :, page * dim // 2:] = blocks[:, :, page * dim // 2:] % 8 + 40      # scales 1/4 to 1/2
    table = torch.randperm(pages, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).int().view(1, -1)
    c = binding.Kv4Cache(pool, torch.tensor([n], dtype=torch.int32, device="cuda"), 1, dim, page, table,
                         torch.zeros(1, 1, pages * page, device="cuda"))
    q = torch.randn(1, 1, 2, dim, generator=torch.Generator().manual_seed(3)).cuda()
    out = _attend(c, q, True)
    k = torch.zeros(1, n, 1, dim, device="cuda")
    v = torch.zeros_like(k)
    binding.kv4_read(c, k, v)
    kd, vd, qd = k[0, :, 0].double(), v[0, :, 0].double(), q[0, 0].double()
    w = torch.softmax(qd @ kd.T / 8, -1)
    want, mass = w @ vd, w @ vd.abs()
    reach = (qd.abs() @ kd.abs().T).amax(-1) / 8
    tol = _bound(want.cpu().numpy(), mass.cpu().numpy(), reach.cpu().numpy(), q.dtype)
    # fp32 sums over 2.6 million keys: 1,100 additions a thread, then 28 partials
    tol = tol + mass.cpu().numpy() * 1200 * 2.0 ** -24
    assert (np.abs((out[0, 0].double() - want).cpu().numpy()) <= tol).all()
    t = 4 * 2.0 ** -18 * float(reach.max()) + 2.0 ** -17 + 1200 * 2.0 ** -24
    assert ((c.scores[0, 0, :n].double() - w.sum(0)).abs() <= w.sum(0) * t + 1e-30).all()


def test_every_operator_is_replayed_from_a_graph(cuda_ok):
    """Append, attention, eviction and reading captured together, replayed with
    other contents, lengths and offsets."""
    p = Plain(2, 2, 64, 32, 3, seed=5)
    c = _cuda(p, [0, 0], np.zeros((2, 2, 96)))
    d = Plain(2, 2, 64, 32, 1, seed=6)
    dst = _cuda(d, [0, 0], np.zeros((2, 2, 32)))
    k, v = torch.zeros(2, 120, 2, 64, device="cuda")
    offs = torch.zeros(3, dtype=torch.int32, device="cuda")
    q = torch.randn(2, 1, 4, 64, generator=torch.Generator().manual_seed(3)).cuda()
    out, ws = torch.zeros_like(q), _workspace(c, 1, 4, True)
    kept = torch.zeros(2, 2, 32, dtype=torch.int32, device="cuda")
    ko, vo = torch.zeros(2, 2, 32, 2, 64, device="cuda")

    def step():
        binding.kv4_append(c, k, v, offs)
        binding.attention_kv4(c, q, out, ws, accumulate=True)
        binding.kv4_evict(c, dst, 32, 2, 3, kept)
        binding.kv4_read(dst, ko, vo)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed, lens in ((1, [60, 60]), (2, [96, 0]), (3, [5, 33])):
        x = torch.randn(2, 120, 2, 64, generator=torch.Generator().manual_seed(seed))
        k.copy_(x[0])
        v.copy_(x[1])
        offs.copy_(torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32))
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        dst.lens.copy_(torch.tensor(lens, dtype=torch.int32).clamp(max=32))
        graph.replay()
        torch.cuda.synchronize()
        for s, a in ((0, 0), (1, lens[0])):
            for j in range(lens[s]):
                p.write(s, j, x[0, a + j].double().numpy(), x[1, a + j].double().numpy())
        _check(p, lens, q, out, 0.125)
        weights = c.scores.cpu().numpy()
        for s, n in enumerate(lens):
            a, b = p.read(s, n)
            for h in range(2):
                want = _kept(weights[s, h], n, 32, 2, 3)
                assert kept[s, h].tolist() == want + [-1] * (32 - len(want))
                assert np.array_equal(ko[s, :len(want), h].double().cpu().numpy(), a[want, h])
                assert np.array_equal(vo[s, :len(want), h].double().cpu().numpy(), b[want, h])


def test_evict_and_append_twice_at_once(cuda_ok):
    """The same call on two streams, caches of their own."""
    n = 9000
    rng = np.random.default_rng(2)
    scores = np.exp(rng.normal(size=(1, 4, 9024)))
    p = Plain(1, 4, 64, 32, 282, seed=1)
    p.fill_random([n])
    src = [_cuda(p, [n], scores) for _ in range(2)]
    d = Plain(1, 4, 64, 32, 32, seed=2)
    dst = [_cuda(d, [1000], np.zeros((1, 4, 1024))) for _ in range(2)]
    kept = [torch.zeros(1, 4, 1000, dtype=torch.int32, device="cuda") for _ in range(2)]
    x = torch.randn(2, 1000, 4, 64, generator=torch.Generator().manual_seed(1)).cuda()
    offs = torch.tensor([0, 1000], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for i in range(2):
        st = torch.cuda.Stream()
        for _ in range(3):
            binding.kv4_append(src[i], x[0], x[1], offs, stream=st)
            binding.kv4_evict(src[i], dst[i], 1000, 4, 32, kept[i], stream=st)
    torch.cuda.synchronize()
    assert torch.equal(kept[0], kept[1]) and torch.equal(dst[0].pool, dst[1].pool)
    sc = src[0].scores.cpu().numpy()
    for h in range(4):
        assert kept[0][0, h].tolist() == _kept(sc[0, h], n, 1000, 4, 32)


def test_the_binding_refuses_other_tensors(cuda_ok):
    pool = torch.zeros(4, binding.kv4_page_bytes(2, 64, 32), dtype=torch.uint8, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad, err in ((dict(pool=pool.cpu()), TypeError), (dict(lens=lens.long()), TypeError), (dict(pool=pool[:3]), ValueError),
                     (dict(pool=pool[:, :-1]), ValueError), (dict(head_dim=96), binding.MkError),
                     (dict(scores=torch.zeros(2, 2, 63, device="cuda")), ValueError),
                     (dict(table=torch.zeros(3, 2, dtype=torch.int32, device="cuda")), ValueError)):
        kw = dict(pool=pool, lens=lens, n_kv_heads=2, head_dim=64, page_tokens=32)
        kw.update(bad)
        with pytest.raises(err):
            binding.Kv4Cache(**kw)
    c = binding.Kv4Cache(pool, lens, 2, 64, 32)
    k = torch.zeros(3, 2, 64, device="cuda")
    offs = torch.zeros(3, dtype=torch.int32, device="cuda")
    for args in ((k, k[:2], offs), (k, k.half(), offs), (k[:, :1], k[:, :1], offs), (k, k, offs[:2]), (k.cpu(), k, offs),
                 (k.transpose(1, 2), k, offs)):
        with pytest.raises(ValueError):
            binding.kv4_append(c, *args)
    with pytest.raises(TypeError):
        binding.kv4_append(c, k.double(), k.double(), offs)
    q = torch.zeros(2, 1, 4, 64, device="cuda")
    ws = _workspace(c, 1, 4, False)
    for args in ((q[:1], q[:1], ws), (q, q[:, :, :2], ws), (q.transpose(2, 3), q, ws)):
        with pytest.raises((ValueError, TypeError)):
            binding.attention_kv4(c, *args)
    with pytest.raises(TypeError):
        binding.attention_kv4(c, q, torch.zeros_like(q).half(), ws)
    with pytest.raises(binding.MkError):                      # a workspace that is too small
        binding.attention_kv4(c, q, torch.zeros_like(q), ws[:4096])
    with pytest.raises(binding.MkError):                      # no scores to add to
        binding.attention_kv4(c, q, torch.zeros_like(q), _workspace(c, 1, 4, True), accumulate=True)


def test_attention_repeats_bit_for_bit_on_other_streams_and_workspaces(cuda_ok):
    lens = [900, 13, 4100]
    p = Plain(3, 4, 128, 64, 65, seed=4)
    p.fill_random(lens)
    q = torch.randn(3, 2, 16, 128, generator=torch.Generator().manual_seed(3)).cuda()
    zero = np.zeros((3, 4, p.capacity))
    a = _cuda(p, lens, zero)
    first = _attend(a, q, True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    caches = [_cuda(p, lens, zero) for _ in streams]
    outs = [torch.empty_like(q) for _ in streams]
    ws = [_workspace(a, 2, 16, True) for _ in streams]
    torch.cuda.synchronize()
    for c, o, w, st in zip(caches, outs, ws, streams):   # two calls at once
        binding.attention_kv4(c, q, o, w, accumulate=True, stream=st)
    torch.cuda.synchronize()
    for c, o in zip(caches, outs):
        assert torch.equal(o, first) and torch.equal(c.scores, a.scores)


def test_attention_graph_replays_with_other_lengths(cuda_ok):
    p = Plain(3, 2, 128, 32, 20, seed=6)
    p.fill_random([640] * 3)
    zero = np.zeros((3, 2, p.capacity))
    c = _cuda(p, [5, 640, 0], zero)
    q = torch.randn(3, 1, 8, 128, generator=torch.Generator().manual_seed(3)).cuda()
    out = torch.empty_like(q)
    ws = _workspace(c, 1, 8, True)
    binding.attention_kv4(c, q, out, ws, accumulate=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.attention_kv4(c, q, out, ws, accumulate=True)
    for lens in ([1, 2, 3], [0, 0, 0], [640, 639, 33]):
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.scores.zero_()
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        _check(p, lens, q, out, 128 ** -0.5, c.scores, zero)


# ---------------------------------------------------------------- eviction

def _kept(scores, n, budget, first, last):
    if n <= budget:
        return list(range(n))
    mid = np.where(np.isnan(scores[first:n - last]), -np.inf, scores[first:n - last])
    take = budget - first - last
    best = np.argsort(-mid, kind="stable")[:take] + first
    return list(range(first)) + sorted(best.tolist()) + list(range(n - last, n))


def _evict_case(p, lens, scores, budget, first, last, page):
    c = _cuda(p, lens, scores)
    per = -(-budget // page)
    rng = np.random.default_rng(1)
    d = Plain(p.n_seq, p.heads, p.dim, page, per, seed=11, n_pages=p.n_seq * per + 3, fill=0x11)
    sc = np.full((p.n_seq, p.heads, d.capacity), -5.0)
    dst = _cuda(d, np.minimum(lens, budget).tolist(), sc)
    kept = torch.full((p.n_seq, p.heads, budget), 99, dtype=torch.int32, device="cuda")
    binding.kv4_evict(c, dst, budget, first, last, kept)
    got = kept.cpu().numpy()
    for s, n in enumerate(lens):
        n = min(max(n, 0), p.capacity)
        for h in range(p.heads):
            want = _kept(scores[s, h], n, budget, first, last)
            assert got[s, h].tolist() == want + [-1] * (budget - len(want)), (s, h)
            for to, slot in enumerate(want):
                pa, a = p._at(s, slot, h)
                pb, b = d._at(s, to, h)
                for w in (0, 1):
                    d.pool[pb, b[w][0]:b[w][0] + d.dim // 2] = p.pool[pa, a[w][0]:a[w][0] + d.dim // 2]
                    d.pool[pb, b[w][1]:b[w][1] + d.dim // GROUP] = p.pool[pa, a[w][1]:a[w][1] + d.dim // GROUP]
                sc[s, h, to] = scores[s, h, slot]
    assert np.array_equal(dst.pool.cpu().numpy(), d.pool)
    assert np.array_equal(dst.scores.cpu().numpy(), sc.astype(np.float32), equal_nan=True)
    assert np.array_equal(c.pool.cpu().numpy(), p.pool)


@pytest.mark.parametrize("lens,heads,dim,page,budget,first,last,to_page", [
    ([1], 1, 64, 32, 1, 0, 0, 32), ([2], 1, 128, 32, 1, 0, 0, 32), ([2], 1, 128, 32, 1, 0, 1, 32),
    ([0, 5, 64, 65, 100], 2, 64, 32, 64, 4, 16, 96), ([100, 300], 3, 128, 64, 33, 0, 0, 32),
    ([500, 90], 2, 64, 64, 90, 40, 50, 64), ([2100, 2048], 2, 64, 64, 1000, 4, 64, 32),
    ([9000, 8191], 1, 64, 64, 4096, 1, 7, 64), ([70, -4, 900], 2, 128, 32, 64, 4, 60, 32),
])
def test_evict_keeps_the_ends_and_the_highest(cuda_ok, lens, heads, dim, page, budget, first, last, to_page):
    p = Plain(len(lens), heads, dim, page, -(-max(lens) // page), seed=budget)
    p.fill_random(lens)
    rng = np.random.default_rng(budget)
    scores = np.exp(2 * rng.normal(size=(len(lens), heads, p.capacity))).astype(np.float32)
    scores[rng.random(scores.shape) < 0.3] = 0.0
    _evict_case(p, lens, scores, budget, first, last, to_page)


@pytest.mark.parametrize("kind", ["equal", "two", "negative", "nan", "infinite", "neighbours"])
@pytest.mark.parametrize("n", [40, 3000])
def test_evict_ties_go_to_the_lowest_slot(cuda_ok, kind, n):
    p = Plain(1, 2, 64, 32, -(-n // 32), seed=1)
    p.fill_random([n])
    rng = np.random.default_rng(3)
    scores = np.full((1, 2, p.capacity), 0.25, np.float32)
    if kind == "two":
        scores[rng.random(scores.shape) < 0.4] = 0.5
    if kind == "negative":
        scores = rng.choice(np.float32([-1.0, -0.0, 0.0, -2.5]), scores.shape)
    if kind == "nan":
        scores[rng.random(scores.shape) < 0.9] = np.nan
    if kind == "infinite":
        scores = rng.choice(np.float32([-np.inf, np.inf, 1.0, np.nan]), scores.shape)
    if kind == "neighbours":
        scores = (np.float32(1.0).view(np.int32) + rng.integers(0, 3, scores.shape)).astype(np.int32).view(np.float32)
    ref = np.where(np.isnan(scores), -np.inf, scores) if kind != "infinite" else scores
    if kind == "infinite":   # NaN below -inf
        ref = scores.copy()
        order = np.where(np.isnan(scores), -3.0, np.where(scores == -np.inf, -2.0, np.where(scores == np.inf, 9.0, 1.0)))
        c = _cuda(p, [n], scores)
        dst = _cuda(Plain(1, 2, 64, 32, 1, seed=2), [25], np.zeros((1, 2, 32)))
        kept = torch.zeros(1, 2, 25, dtype=torch.int32, device="cuda")
        binding.kv4_evict(c, dst, 25, 2, 3, kept)
        for h in range(2):
            assert kept[0, h].tolist() == _kept(order[0, h], n, 25, 2, 3)
        return
    _evict_case(p, [n], scores, 25, 2, 3, 32)


def test_evict_longer_than_the_registers(cuda_ok):
    """More keys than one pass holds (32,768): the threshold and the order go
    over several, with ties on the border in each."""
    n = 70001
    p = Plain(1, 1, 64, 64, -(-n // 64), seed=1)
    p.pool[:] = np.random.default_rng(0).integers(0, 119, p.pool.shape)
    rng = np.random.default_rng(5)
    scores = np.exp(rng.normal(size=(1, 1, p.capacity))).astype(np.float32)
    scores[rng.random(scores.shape) < 0.5] = 1.0
    for budget in (20000, 60000, 70000):
        c = _cuda(p, [n], scores)
        d = Plain(1, 1, 64, 64, -(-budget // 64), seed=2)
        dst = _cuda(d, [budget], np.zeros((1, 1, d.capacity)))
        kept = torch.zeros(1, 1, budget, dtype=torch.int32, device="cuda")
        binding.kv4_evict(c, dst, budget, 4, 100, kept)
        assert np.array_equal(kept[0, 0].cpu().numpy(), _kept(scores[0, 0], n, budget, 4, 100))


def test_evict_with_missing_pages(cuda_ok):
    """A kept slot without a page leaves its place; a destination without one
    is not written."""
    p = Plain(1, 1, 64, 32, 3, seed=1)
    p.fill_random([96])
    p.table[0, 1] = -1
    scores = np.arange(96, dtype=np.float32).reshape(1, 1, 96)
    c = _cuda(p, [96], scores)
    d = Plain(1, 1, 64, 32, 2, seed=2, fill=0x55)
    d.table[0, 1] = 1000
    dst = _cuda(d, [64], np.zeros((1, 1, 64)))
    kept = torch.zeros(1, 1, 64, dtype=torch.int32, device="cuda")
    binding.kv4_evict(c, dst, 64, 8, 0, kept)
    want = _kept(scores[0, 0], 96, 64, 8, 0)
    assert kept[0, 0].tolist() == want
    for to, slot in enumerate(want[:32]):
        if slot // 32 == 1:
            continue
        pa, a = p._at(0, slot, 0)
        pb, b = d._at(0, to, 0)
        for w in (0, 1):
            d.pool[pb, b[w][0]:b[w][0] + 32] = p.pool[pa, a[w][0]:a[w][0] + 32]
            d.pool[pb, b[w][1]:b[w][1] + 4] = p.pool[pa, a[w][1]:a[w][1] + 4]
    assert np.array_equal(dst.pool.cpu().numpy(), d.pool)


@pytest.mark.parametrize("dim,page,to_page", [(64, 32, 64), (128, 64, 32)])
def test_attention_after_an_eviction_sees_the_kept_rows_only(cuda_ok, dim, page, to_page):
    """Every slot below lens has a page, as an eviction asks for; the
    destination's pages held NaN before.  Longer, equal, shorter and empty
    sequences; every KV head keeps slots of its own."""
    lens, heads, group, budget = [300, 64, 65, 10, 0], 3, 2, 64
    p = Plain(5, heads, dim, page, -(-300 // page), seed=4)
    p.fill_random(lens)
    scores = np.exp(2 * np.random.default_rng(1).normal(size=(5, heads, p.capacity))).astype(np.float32)
    c = _cuda(p, lens, scores)
    d = Plain(5, heads, dim, to_page, -(-budget // to_page), seed=5, fill=0xFF)
    now = [min(n, budget) for n in lens]
    dst = _cuda(d, now, np.full((5, heads, d.capacity), np.nan))
    kept = torch.zeros(5, heads, budget, dtype=torch.int32, device="cuda")
    binding.kv4_evict(c, dst, budget, 4, 16, kept)
    q = torch.randn(5, 2, heads * group, dim, generator=torch.Generator().manual_seed(2)).cuda()
    out = _attend(dst, q, True)
    got = kept.cpu().numpy()
    for s, n in enumerate(lens):
        k, v = p.read(s, n)
        at = got[s, :, :now[s]].T                                      # [slots][heads]
        k, v = (np.take_along_axis(x, at[..., None], 0) for x in (k, v))
        want, w, mass, reach = attend(q[s].double().cpu().numpy(), k, v, dim ** -0.5, group)
        assert (np.abs(out[s].double().cpu().numpy() - want) <= _bound(want, mass, reach, q.dtype)).all()
        before = np.take_along_axis(scores[s].astype(np.float64), at.T, 1)
        t = 4 * 2.0 ** -18 * (reach.max() if reach.size else 0) + 2.0 ** -17
        after = dst.scores[s, :, :now[s]].double().cpu().numpy()
        assert (np.abs(after - before - w) <= w * t + (before + w) * 2.0 ** -22 + 1e-30).all()


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("captured", [False, True])
def test_a_decode_on_a_budget(cuda_ok, captured):
    """Prompts in, then steps of append and attention, the cache cut back to a
    budget whenever it reaches a limit; every output against the reference
    on the same kept keys, each step eager or replayed from one graph."""
    heads, group, dim, page, budget, limit, steps = 2, 4, 64, 32, 48, 64, 40
    prompts = [50, 3, 64]
    n_seq = len(prompts)
    rng = np.random.default_rng(7)
    plains = [Plain(n_seq, heads, dim, page, 2, seed=s) for s in (1, 2)]
    caches = [_cuda(p, prompts, np.zeros((n_seq, heads, 64))) for p in plains]
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    for c in caches:
        c.lens.copy_(lens)
    x = rng.normal(size=(2, sum(prompts), heads, dim)).astype(np.float32)
    offs = torch.tensor(np.cumsum([0] + prompts), dtype=torch.int32, device="cuda")
    kt, vt = torch.from_numpy(x).cuda()
    binding.kv4_append(caches[0], kt, vt, offs)
    rows = [[x[:, o:o + n] for o, n in zip(np.cumsum([0] + prompts), prompts)]][0]
    for s, r in enumerate(rows):
        for j in range(r.shape[1]):
            plains[0].write(s, j, r[0, j], r[1, j])
    assert np.array_equal(caches[0].pool.cpu().numpy(), plains[0].pool)
    one = torch.arange(n_seq + 1, dtype=torch.int32, device="cuda")
    k1, v1 = torch.zeros(2, n_seq, heads, dim, device="cuda")
    q = torch.zeros(n_seq, 1, heads * group, dim, device="cuda")
    out = torch.zeros_like(q)
    ws = _workspace(caches[0], 1, heads * group, True)
    kept = torch.zeros(n_seq, heads, budget, dtype=torch.int32, device="cuda")

    def step(c):
        binding.kv4_append(c, k1, v1, one)
        binding.attention_kv4(c, q, out, ws, accumulate=True)

    graphs = [None, None]
    if captured:
        for i, c in enumerate(caches):
            saved = c.pool.clone(), c.scores.clone()
            step(c)
            torch.cuda.synchronize()
            graphs[i] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[i]):
                step(c)
            c.pool.copy_(saved[0])
            c.scores.copy_(saved[1])
    cur, now = 0, list(prompts)
    for s, r in enumerate(rows):
        rows[s] = [r[:, j] for j in range(r.shape[1])]
    for i in range(steps):
        if max(now) == limit:
            before = caches[cur].scores.cpu().numpy()
            binding.kv4_evict(caches[cur], caches[1 - cur], budget, 4, 8, kept)
            got = kept.cpu().numpy()
            for s in range(n_seq):
                for h in range(heads):
                    want = _kept(before[s, h], now[s], budget, 4, 8)
                    assert [a for a in got[s, h].tolist() if a >= 0] == want
                    for to, slot in enumerate(want):
                        pa, a = plains[cur]._at(s, slot, h)
                        pb, b = plains[1 - cur]._at(s, to, h)
                        for w in (0, 1):
                            plains[1 - cur].pool[pb, b[w][0]:b[w][0] + dim // 2] = plains[cur].pool[pa, a[w][0]:a[w][0] + dim // 2]
                            plains[1 - cur].pool[pb, b[w][1]:b[w][1] + dim // 16] = plains[cur].pool[pa, a[w][1]:a[w][1] + dim // 16]
            now = [min(n, budget) for n in now]
            cur = 1 - cur
        now = [n + 1 for n in now]
        caches[cur].lens.copy_(torch.tensor(now, dtype=torch.int32))
        new = rng.normal(size=(2, n_seq, heads, dim)).astype(np.float32)
        k1.copy_(torch.from_numpy(new[0]))
        v1.copy_(torch.from_numpy(new[1]))
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(i)))
        before = caches[cur].scores.cpu().numpy().astype(np.float64)
        if captured:
            graphs[cur].replay()
        else:
            step(caches[cur])
        for s in range(n_seq):
            plains[cur].write(s, now[s] - 1, new[0, s], new[1, s])
            before[s, :, now[s] - 1] = 0.0
        _check(plains[cur], now, q, out, dim ** -0.5, caches[cur].scores, before)
    assert cur == 1 or steps < limit - max(prompts)


def test_prefix_pages_shared_by_sequences(cuda_ok):
    """Two sequences read one prompt's page; each appends to pages of its own."""
    p = Plain(2, 2, 128, 32, 2, seed=2)
    p.table[1, 0] = p.table[0, 0]
    p.fill_random([64, 64])
    lens = [40, 50]
    q = torch.randn(2, 1, 8, 128, generator=torch.Generator().manual_seed(3)).cuda()
    c = _cuda(p, lens)
    _check(p, lens, q, _attend(c, q), 128 ** -0.5)
