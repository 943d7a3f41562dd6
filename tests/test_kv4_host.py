"""The operators on a decode's state refuse bad arguments before they touch a
device (addresses here are never dereferenced), and their sizes are what the
format says."""
import ctypes as C
import math

import pytest
import torch

from persistent_megakernel_03_b200 import binding

A = 0x10000   # an aligned address that nobody reads


def _cache(**kw):
    f = dict(n_kv_heads=2, head_dim=64, page_tokens=64, n_pages=8, n_seq=2, pages_per_seq=4, k_log2=0,
             v_log2=0, pool_dev=A, table_dev=A, lens_dev=A, scores_dev=A)
    f.update(kw)
    return binding.Kv4Struct(*[f[n] for n, _ in binding.Kv4Struct._fields_])


def _refused(rc, code, part):
    L = binding.lib()
    assert rc == code, rc
    msg = L.mk_last_error(None).decode()
    assert part in msg, msg


BAD_CACHES = [
    (dict(pool_dev=None), -1, "pool"), (dict(lens_dev=None), -1, "lengths"), (dict(head_dim=96), -9, "head_dim"),
    (dict(n_kv_heads=0), -1, "n_kv_heads"), (dict(n_kv_heads=1025), -1, "n_kv_heads"),
    (dict(page_tokens=0), -1, "page_tokens"), (dict(page_tokens=48), -1, "page_tokens"),
    (dict(n_seq=0), -1, "n_seq"), (dict(n_seq=4097), -1, "n_seq"), (dict(n_pages=0), -1, "n_pages"),
    (dict(pages_per_seq=0), -1, "pages_per_seq"), (dict(pages_per_seq=1 << 25), -1, "2^30"),
    (dict(table_dev=None, n_pages=7), -1, "without a table"), (dict(k_log2=33), -1, "k_log2"),
    (dict(v_log2=-33), -1, "v_log2"), (dict(pool_dev=A + 8), -1, "16-byte"), (dict(lens_dev=A + 2), -1, "4-byte"),
]


@pytest.mark.parametrize("change,code,part", BAD_CACHES)
def test_every_operator_checks_its_cache(change, code, part):
    L, c, ok = binding.lib(), _cache(**change), _cache()
    r, good = C.addressof(c), C.addressof(ok)
    _refused(L.mk_kv4_append(r, A, A, 0, 128, 128, A, 1, None), code, part)
    _refused(L.mk_kv4_read(r, 0, 1, A, A, None), code, part)
    _refused(L.mk_attention_kv4(r, A, 0, 1, 4, 256, 1.0, 0, A, 1 << 40, A, None), code, part)
    _refused(L.mk_kv4_evict(r, good, 1, 0, 0, A, None), code, part)
    _refused(L.mk_kv4_evict(good, r, 1, 0, 0, A, None), code, part)
    _refused(L.mk_kv4_reorder(r, A, 2, 0, 1, None), code, part)
    assert L.mk_attention_kv4_workspace_bytes(r, 1, 4, 0) == 0


def test_no_cache():
    L = binding.lib()
    _refused(L.mk_kv4_append(None, A, A, 0, 128, 128, A, 1, None), -1, "no cache")
    assert L.mk_attention_kv4_workspace_bytes(None, 1, 4, 0) == 0


@pytest.mark.parametrize("args,part", [
    ((A, A, 3, 128, 128, A, 1), "dtype"), ((A, A, 0, 128, 128, A, -1), "n_tokens"), ((A, A, 0, 128, 128, A, (1 << 30) + 1), "n_tokens"), ((A, A, 0, 128, 128, None, 1), "offsets"),
    ((None, A, 0, 128, 128, A, 1), "keys"), ((A, None, 0, 128, 128, A, 1), "keys"), ((A, A, 0, 127, 128, A, 1), "stride"),
    ((A, A, 0, 128, 64, A, 1), "stride"), ((A + 4, A, 0, 128, 128, A, 1), "aligned"), ((A, A, 1, 132, 128, A, 1), "aligned"),
    ((A, A, 0, 128, 130, A, 1), "aligned"),
])
def test_append_refuses(args, part):
    c = _cache()
    _refused(binding.lib().mk_kv4_append(C.addressof(c), *args, None), -1, part)


def test_append_refuses_offsets_between_words():
    c = _cache()
    _refused(binding.lib().mk_kv4_append(C.addressof(c), A, A, 0, 128, 128, A + 2, 1, None), -1, "offsets")


def test_empty_calls_are_no_errors():
    L, c = binding.lib(), _cache()
    r = C.addressof(c)
    assert L.mk_kv4_append(r, None, None, 0, 128, 128, A, 0, None) == 0
    assert L.mk_kv4_read(r, 0, 0, None, None, None) == 0
    assert L.mk_kv4_reorder(r, A, 2, 5, 5, None) == 0
    assert L.mk_kv4_reorder(r, A, 1, 0, 5, None) == 0
    assert L.mk_beam_reorder(A, A, 2, 1, 64, 1, 64, 64, None) == 0
    assert L.mk_beam_reorder(A, A, 2, 2, 64, 0, 64, 64, None) == 0


@pytest.mark.parametrize("args,part", [
    ((3, 1, A, A), "dtype"), ((0, -1, A, A), "negative"), ((0, 1, None, A), "outputs"), ((0, 1, A, A + 8), "aligned")])
def test_read_refuses(args, part):
    c = _cache()
    _refused(binding.lib().mk_kv4_read(C.addressof(c), *args, None), -1, part)


@pytest.mark.parametrize("change,part", [
    (dict(q_len=0), "q_len"), (dict(q_len=513), "q_len"), (dict(heads=0), "n_q_heads"), (dict(heads=3), "n_q_heads"),
    (dict(dtype=3), "dtype"), (dict(q=None), "queries"), (dict(out=None), "queries"), (dict(stride=255), "stride"),
    (dict(q=A + 8), "aligned"), (dict(dtype=1, stride=260), "aligned"), (dict(out=A + 2), "aligned"),
    (dict(scale=0.0), "scale"), (dict(scale=-1.0), "scale"), (dict(scale=float("nan")), "scale"),
    (dict(scale=float("inf")), "scale"), (dict(scale=1e-19), "scale"), (dict(scale=2e18), "scale"), (dict(ws=None), "workspace"), (dict(ws=A + 4), "workspace"),
    (dict(size=-1), "workspace"),
])
def test_attention_refuses(change, part):
    L, c = binding.lib(), _cache()
    f = dict(q=A, dtype=0, q_len=1, heads=4, stride=256, scale=1.0, acc=0, ws=A, size=0, out=A)
    f.update(change)
    need = L.mk_attention_kv4_workspace_bytes(C.addressof(c), 1, 4, 0)
    assert need > 0
    _refused(L.mk_attention_kv4(C.addressof(c), f["q"], f["dtype"], f["q_len"], f["heads"], f["stride"], f["scale"],
                                f["acc"], f["ws"], need + f["size"], f["out"], None), -1, part)


def test_attention_accumulates_only_into_scores():
    c = _cache(scores_dev=None)
    _refused(binding.lib().mk_attention_kv4(C.addressof(c), A, 0, 1, 4, 256, 1.0, 1, A, 1 << 40, A, None), -1, "scores")


def test_workspace_grows_with_what_it_holds():
    L = binding.lib()
    small, long = _cache(), _cache(pages_per_seq=400, n_pages=800)
    plain = L.mk_attention_kv4_workspace_bytes(C.addressof(small), 1, 4, 0)
    assert plain == L.mk_attention_kv4_workspace_bytes(C.addressof(long), 1, 4, 0)
    # scores of 2 rows (4 query heads on 2 KV heads) of every slot, fp32
    more = L.mk_attention_kv4_workspace_bytes(C.addressof(long), 1, 4, 1)
    assert more >= plain + 2 * 2 * 400 * 64 * 2 * 4
    # 34 rows of every slot at least
    more = L.mk_attention_kv4_workspace_bytes(C.addressof(long), 17, 4, 1)
    assert more >= 2 * 2 * 34 * 400 * 64 * 4


@pytest.mark.parametrize("src,dst,args,part", [
    ({}, dict(n_kv_heads=3), (1, 0, 0, A), "both"), ({}, dict(head_dim=128), (1, 0, 0, A), "both"),
    ({}, dict(n_seq=1), (1, 0, 0, A), "both"), ({}, dict(k_log2=1), (1, 0, 0, A), "both"),
    (dict(scores_dev=None), {}, (1, 0, 0, A), "scores"), ({}, {}, (0, 0, 0, A), "budget"),
    ({}, dict(pages_per_seq=1), (65, 0, 0, A), "budget"), ({}, {}, (8, 5, 4, A), "keep_first"),
    ({}, {}, (8, -1, 4, A), "keep_first"), ({}, {}, (8, 1, 4, None), "kept"), ({}, {}, (8, 1, 4, A + 1), "kept"),
    ({}, dict(pool_dev=A), (8, 1, 4, A), "of its own"), ({}, dict(scores_dev=A), (8, 1, 4, A), "of its own"),
])
def test_evict_refuses(src, dst, args, part):
    d = dict(pool_dev=2 * A, scores_dev=3 * A)
    d.update(dst)
    a, b = _cache(**src), _cache(**d)
    _refused(binding.lib().mk_kv4_evict(C.addressof(a), C.addressof(b), *args, None), -1, part)


@pytest.mark.parametrize("args,part", [
    ((A, 0, 0, 1), "beams"), ((A, 17, 0, 1), "beams"), ((A, 3, 0, 1), "searches"), ((A, 2, -1, 1), "first"),
    ((A, 2, 3, 2), "first"), ((A, 2, 0, 257), "first"), ((None, 2, 0, 1), "parents"), ((A + 1, 2, 0, 1), "parents")])
def test_kv4_reorder_refuses(args, part):
    c = _cache()
    _refused(binding.lib().mk_kv4_reorder(C.addressof(c), *args, None), -1, part)


SELECT = dict(logits=A, dtype=0, stride=1000, cum=A, fin=None, n=2, beams=4, vocab=1000, eos=-1, tok=2 * A, par=3 * A,
              sc=4 * A, done=None, ws=A, size=0)


@pytest.mark.parametrize("change,part", [
    (dict(n=0), "rows"), (dict(beams=0), "beams"), (dict(beams=17), "beams"), (dict(n=20000), "rows"),
    (dict(vocab=0), "vocab"), (dict(vocab=1048577, stride=1048577), "vocab"), (dict(dtype=4), "dtype"),
    (dict(logits=None), "wanted"), (dict(cum=None), "wanted"), (dict(tok=None), "wanted"), (dict(sc=None), "wanted"),
    (dict(stride=999), "apart"), (dict(eos=1000), "eos"), (dict(eos=-2), "eos"), (dict(fin=A), "eos"),
    (dict(fin=A, done=A, eos=1), "two arrays"), (dict(sc=A), "two arrays"), (dict(logits=A + 2), "aligned"),
    (dict(par=A + 1), "aligned"), (dict(ws=None), "workspace"), (dict(ws=A + 8), "workspace"), (dict(size=-1), "workspace"),
])
def test_select_refuses(change, part):
    L, f = binding.lib(), dict(SELECT)
    f.update(change)
    need = L.mk_beam_select_workspace_bytes(2, 4, 1000)
    assert need == 2 * 4 * (8 + 4 * 8)
    _refused(L.mk_beam_select(f["logits"], f["dtype"], f["stride"], f["cum"], f["fin"], f["n"], f["beams"], f["vocab"],
                              f["eos"], f["tok"], f["par"], f["sc"], f["done"], f["ws"], need + f["size"], None), -1, part)


@pytest.mark.parametrize("change,part", [
    (dict(n=0), "searches"), (dict(n=32768), "searches"), (dict(beams=17), "beams"), (dict(segs=-1), "segments"),
    (dict(segs=65536), "segments"), (dict(state=None), "state"), (dict(par=None), "state"), (dict(state=A + 8), "16"),
    (dict(beam=264), "16"), (dict(seg=72), "16"), (dict(size=40), "16"), (dict(par=A + 2), "4-byte"),
    (dict(size=80), "overlap"), (dict(beam=192), "overlap"), (dict(beam=0), "overlap"),
])
def test_reorder_refuses(change, part):
    f = dict(state=A, par=A, n=2, beams=2, beam=256, segs=4, seg=64, size=64)
    f.update(change)
    _refused(binding.lib().mk_beam_reorder(f["state"], f["par"], f["n"], f["beams"], f["beam"], f["segs"], f["seg"],
                                           f["size"], None), -1, part)


@pytest.mark.parametrize("shape,strides", [
    ((4, 2, 3, 8), (48, 24, 8, 1)), ((4, 1, 1, 16), (16, 999, 777, 1)), ((4, 1, 1, 16), (16, 1, 1, 1)),
    ((4, 3, 1, 16), (48, 16, 4096, 1)), ((4, 1, 5), (5, 64, 1))])
def test_binding_reorder_goes_by_shape(shape, strides, monkeypatch):
    """The stride of an axis of one entry means nothing: such a tensor is contiguous."""
    seen = []
    monkeypatch.setattr(binding, "_tensor", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(binding, "_on", lambda device, stream, call, *a: seen.append(a))
    state = torch.empty(200).as_strided(shape, strides)
    assert state.is_contiguous()
    n = shape[2]
    binding.beam_reorder(state, torch.zeros(2, 2, dtype=torch.int32), n - 1, 1)
    row = 4 * math.prod(shape[3:])
    assert seen[0][0] == state.data_ptr() + (n - 1) * row
    assert seen[0][2:] == (2, 2, shape[1] * n * row, shape[1], n * row, row)


def test_reorder_takes_beams_inside_segments():
    """[segment][row]: rows a segment's bytes apart, segments all rows apart."""
    L = binding.lib()
    # one beam: checked, and nothing to launch
    assert L.mk_beam_reorder(A, A, 4, 1, 64, 4, 256, 64, None) == 0
    _refused(L.mk_beam_reorder(A, A, 4, 1, 64, 4, 240, 64, None), -1, "overlap")


@pytest.mark.parametrize("heads,dim,page,want", [
    (1, 64, 32, 2304), (8, 128, 64, 73728), (2, 64, 96, 13824), (0, 64, 32, 0), (1, 96, 32, 0), (1, 64, 16, 0),
    (1, 64, 0, 0), (1, 64, 33, 0)])
def test_page_bytes(heads, dim, page, want):
    assert binding.kv4_page_bytes(heads, dim, page) == want


def test_context_reorder_needs_a_context():
    assert binding.lib().mk_kv_reorder(None, None, 1, A, 0, 1) == -1
