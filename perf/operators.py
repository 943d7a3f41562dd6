"""Cases of the operators that hold the state of a decode: the 4-bit KV cache
(append, read, attention, eviction by accumulated attention weight) and beam
search (selection over beams and vocabulary, reordering of the beams' states).

Each case is one pass as a decoding program makes it:

  attend  attention of the newest q_len tokens of every sequence over its cache
  step    append of the newest tokens, then that attention, per layer and step
  prompt  append of packed prompts, and the cache's values read back
  evict   the highest accumulated weights kept in other pages, and read back
  beam    selection of the next beams, and their states moved behind them

The cache's bytes: groups of 16 dims share an e4m3 scale, codes are e2m1, two
per byte (the even dim in the low nibble).  A block is 32 keys of one KV head:
K codes [32][d/2], K scales [32][d/16], V codes, V scales; a page is
[n_kv_heads][page_tokens / 32] blocks.

``run`` computes the plain forms in elementary torch operations, or, where
``own`` is true, calls the package.
"""
import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BLOCK = 32   # keys of a block
GROUP = 16   # dims that share a scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases

def _attend(name, kind, n_seq, lo, hi, kv_heads, group, dim, q_len, dtype, accumulate, page):
    return {"name": name, "kind": kind, "n_seq": n_seq, "lo": lo, "hi": hi, "kv_heads": kv_heads,
            "group": group, "dim": dim, "q_len": q_len, "dtype": dtype, "accumulate": accumulate,
            "page": page}


def _prompt(name, n_seq, lo, hi, kv_heads, dim, dtype, page):
    return {"name": name, "kind": "prompt", "n_seq": n_seq, "lo": lo, "hi": hi,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "page": page}


def _evict(name, n_seq, lo, hi, kv_heads, dim, budget, first, last, page):
    return {"name": name, "kind": "evict", "n_seq": n_seq, "lo": lo, "hi": hi,
            "kv_heads": kv_heads, "dim": dim, "budget": budget, "first": first, "last": last,
            "page": page}


def _beam(name, n_batch, beams, vocab, dtype, segments, positions, first, count, dim):
    return {"name": name, "kind": "beam", "n_batch": n_batch, "beams": beams, "vocab": vocab,
            "dtype": dtype, "segments": segments, "positions": positions, "first": first,
            "count": count, "dim": dim}


def listed():
    return [
        # the Qwen2.5-0.5B shape at the end of its 39 + 512 workload: one request, latency
        _attend("qwen 1x551 fp32", "attend", 1, 551, 551, 2, 7, 64, 1, "fp32", False, 0),
        # the Llama-3-8B shape's 32K context, weights accumulated for a later eviction
        _attend("llama 1x32768 bf16 acc", "attend", 1, 32768, 32768, 8, 4, 128, 1, "bf16", True, 64),
        # its eight ragged requests (32 to 2048 tokens and 256 steps), the whole step of a layer
        _attend("llama 8 ragged fp32 step", "step", 8, 32, 2304, 8, 4, 128, 1, "fp32", True, 64),
        # a serving batch of long requests
        _attend("llama 64x8191 bf16", "attend", 64, 6001, 8191, 8, 4, 128, 1, "bf16", False, 128),
        # five draft tokens checked at once, requests from empty to long
        _attend("verify 16x5 tokens fp16", "step", 16, 3, 4097, 8, 4, 128, 5, "fp16", False, 64),
        # eight packed prompts of the Llama-3-8B shape enter the cache
        _prompt("prompts 8 ragged bf16", 8, 32, 2048, 8, 128, "bf16", 64),
        # one short prompt of the Qwen2.5-0.5B shape, in the decoder's own type
        _prompt("prompt 1x39 fp32", 1, 39, 39, 2, 64, "fp32", 0),
        # a long prompt's cache cut to a budget once the prompt is in
        _evict("evict 32768 to 4096", 1, 32768, 32768, 8, 128, 4096, 4, 256, 64),
        # a serving batch that ran some steps past its budget
        _evict("evict 16 ragged to 1024", 16, 700, 1153, 2, 64, 1024, 4, 64, 64),
        # the tiny decoder: selection is all latency
        _beam("beam 1x4 of 4096 fp32", 1, 4, 4096, "fp32", 8, 32, 16, 16, 64),
        # eight hypotheses of the Llama-3-8B shape, their generated positions moved
        _beam("beam 1x8 of 128256 fp32", 1, 8, 128256, "fp32", 512, 551, 39, 256, 128),
        # a batch of searches with the Qwen2.5-0.5B shape's vocabulary
        _beam("beam 16x4 of 151936 bf16", 16, 4, 151936, "bf16", 96, 160, 39, 101, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("attend", "attend", "step", "prompt", "evict", "beam"))
    if kind == "beam":
        vocab = _log(rng, 100, 151936)
        beams = rng.randint(1, 16)
        n_batch = _log(rng, 1, max(1, min(64, 10_000_000 // (vocab * beams))))
        dim = rng.choice((64, 128))
        positions = _log(rng, 8, 512)
        first = rng.randint(0, positions - 1)
        room = 250_000_000 // (n_batch * beams * positions * dim * 2)
        c = _beam("", n_batch, beams, vocab, rng.choice(tuple(DTYPES)),
                  _log(rng, 1, max(1, min(512, room))), positions, first,
                  rng.randint(1, positions - first), dim)
    else:
        kv_heads, group = rng.choice(((1, 8), (2, 7), (2, 2), (4, 1), (8, 4), (8, 8), (4, 16), (3, 5)))
        dim = rng.choice((64, 128))
        n_seq = _log(rng, 1, 64)
        q_len = rng.choice((1, 1, 1, rng.randint(2, 16)))
        most = 16_000_000 // max(1, q_len * group // 24) if kind in ("attend", "step") else 1_000_000
        hi = _log(rng, 1, max(1, min(32768, most // (n_seq * kv_heads * dim // 16))))
        lo = rng.randint(0, hi)
        page = rng.choice((0, 32, 64, 128, 256))
        dtype = rng.choice(tuple(DTYPES))
        if kind == "prompt":
            c = _prompt("", n_seq, lo, hi, kv_heads, dim, dtype, page)
        elif kind == "evict":
            budget = _log(rng, 1, hi + 7)
            first = rng.randint(0, min(8, budget))
            c = _evict("", n_seq, lo, hi, kv_heads, dim, budget, first,
                       rng.randint(0, min(256, budget - first)), page)
        else:
            c = _attend("", kind, n_seq, lo, hi, kv_heads, group, dim, q_len, dtype,
                        rng.random() < 0.5, page)
    del c["name"]
    return c


def _lens(case):
    """Keys of each sequence: a property of the case, the longest and the shortest among them."""
    rng = random.Random("%s" % sorted((k, v) for k, v in case.items() if k != "name"))
    got = [case["hi"], case["lo"]] + [rng.randint(case["lo"], case["hi"]) for _ in range(case["n_seq"])]
    return got[:case["n_seq"]]


def work(case):
    if case["kind"] == "beam":
        size = torch.empty((), dtype=DTYPES[case["dtype"]]).element_size()
        rows, w = case["n_batch"] * case["beams"], case["beams"]
        logits = rows * case["vocab"]
        # of the beams' states, as random parents move them: all but one in W are written, from
        # 1 - (1 - 1/W)^W of them
        state = rows * case["segments"] * case["count"] * case["dim"] * 2
        moved = state * (1 - 1 / w) + state * (1 - (1 - 1 / w) ** w if w > 1 else 0)
        return {"bytes": logits * size + rows * 20 + moved, "flops": 4 * logits}
    heads, dim, lens = case["kv_heads"], case["dim"], _lens(case)
    row = dim + dim // 8                      # bytes of a key and its value in the cache
    if case["kind"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens) * heads
        return {"bytes": sum(lens) * heads * 4 + kept * (3 * row + 2 * 2 * dim + 4 + 4),
                "flops": sum(lens) * heads + kept * 2 * dim}
    size = torch.empty((), dtype=DTYPES[case["dtype"]]).element_size()
    if case["kind"] == "prompt":
        return {"bytes": sum(lens) * heads * (2 * dim * size + 2 * row + 2 * 2 * dim),
                "flops": sum(lens) * heads * 2 * dim * 4}
    q_heads = heads * case["group"]
    rows = case["n_seq"] * case["q_len"]
    b = sum(lens) * heads * (row + (8 if case["accumulate"] else 0)) + 2 * rows * q_heads * dim * size
    if case["kind"] == "step":
        b += sum(min(n, case["q_len"]) for n in lens) * heads * 2 * dim * size
    return {"bytes": b, "flops": 4 * case["q_len"] * q_heads * dim * sum(lens)}


# ------------------------------------------------- the cache's bytes, plainly

def _quantize(x):
    """x [..., dim] -> (bytes of codes [..., dim / 2], bytes of scales [..., dim / 16])."""
    g = x.float().unflatten(-1, (-1, GROUP))
    top = g.abs().amax(-1, keepdim=True)
    # divided by a tensor: a number is turned into its rounded reciprocal, which misses ties
    scale = (top / torch.full_like(top, 6)).clamp(max=448).to(torch.float8_e4m3fn)
    s = scale.float()
    a = g.abs()
    # halfway between two values goes to the even code
    code = ((a > 0.25 * s).byte() + (a >= 0.75 * s).byte() + (a > 1.25 * s).byte() + (a >= 1.75 * s).byte()
            + (a > 2.5 * s).byte() + (a >= 3.5 * s).byte() + (a > 5 * s).byte())
    code = torch.where(s > 0, code, torch.zeros_like(code)) + 8 * (g < 0).byte()
    code = code.flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], scale.squeeze(-1).view(torch.uint8)


def _regions(pool, heads, dim):
    """Views of a pool's K codes, K scales, V codes and V scales: [pages][heads][blocks][32][bytes]."""
    size = BLOCK * (dim + dim // 8)
    blocks = pool.view(pool.shape[0], heads, -1, size)
    got, at = [], 0
    for width in (dim // 2, dim // GROUP, dim // 2, dim // GROUP):
        got.append(blocks[..., at:at + BLOCK * width].unflatten(-1, (BLOCK, width)))
        at += BLOCK * width
    return got


def _store(pool, table, page, heads, dim, seq, slot, k, v):
    """Rows k, v [tokens][heads][dim] into slots `slot` of sequences `seq`."""
    at = table[seq, slot // page].long()
    block, row = slot % page // BLOCK, slot % BLOCK
    kc, ks, vc, vs = _regions(pool, heads, dim)
    for codes, scales, x in ((kc, ks, k), (vc, vs, v)):
        c, s = _quantize(x)
        codes[at, :, block, row] = c
        scales[at, :, block, row] = s


def _values(pool, table, page, heads, dim, keys):
    """Values of slots [0, keys) of every sequence: k, v [n_seq][heads][keys][dim], fp32."""
    pages = -(-keys // page)
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=pool.device)
    got = []
    parts = _regions(pool[table[:, :pages].long()].flatten(0, 1), heads, dim)
    for codes, scales in (parts[:2], parts[2:]):
        c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
        x = lut[c.int()].unflatten(-1, (-1, GROUP)) * scales.contiguous().view(torch.float8_e4m3fn).float().unsqueeze(-1)
        x = x.flatten(-2).flatten(2, 3).unflatten(0, (-1, pages))   # [n_seq][pages][heads][page][dim]
        got.append(x.transpose(1, 2).flatten(2, 3)[:, :, :keys])
    return got


# ------------------------------------------------------------------ inputs

def _keys_values(gen, n, heads, dim, dtype):
    """Keys with channels of unequal size and an offset, as rotated keys have them, and values."""
    dev = "cuda"
    size = torch.exp(0.5 * torch.randn(heads, dim, device=dev, generator=gen))
    off = 0.5 * torch.randn(heads, dim, device=dev, generator=gen)
    k = torch.randn(n, heads, dim, device=dev, generator=gen) * size + off
    v = torch.randn(n, heads, dim, device=dev, generator=gen)
    return k.to(dtype), v.to(dtype)


def _pages(gen, n_seq, most, page):
    """(positions per page, pages, table): pages in random order, or one page for each sequence."""
    page = page or max(BLOCK, -(-most // BLOCK) * BLOCK)
    per = max(1, -(-most // page))
    if per == 1:
        return page, n_seq, torch.arange(n_seq, device="cuda", dtype=torch.int32).view(n_seq, 1)
    return page, n_seq * per, torch.randperm(n_seq * per, device="cuda", generator=gen).int().view(n_seq, per)


def _filled(gen, case, lens):
    """A pool that holds `lens` keys of each sequence, and its table."""
    heads, dim, n_seq = case["kv_heads"], case["dim"], case["n_seq"]
    page, pages, table = _pages(gen, n_seq, max(lens), case["page"])
    pool = torch.zeros(pages, heads * page * (dim + dim // 8), dtype=torch.uint8, device="cuda")
    for s, n in enumerate(lens):
        if n:
            slot = torch.arange(n, device="cuda")
            k, v = _keys_values(gen, n, heads, dim, torch.float32)
            _store(pool, table, page, heads, dim, torch.full_like(slot, s), slot, k, v)
    return page, pool, table


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    if case["kind"] == "beam":
        rows, vocab, w = case["n_batch"] * case["beams"], case["vocab"], case["beams"]
        s["logits"] = (3 * torch.randn(rows, vocab, device="cuda", generator=gen)).to(DTYPES[case["dtype"]])
        # tokens that a grammar forbids
        s["logits"].masked_fill_(torch.rand(rows, vocab, device="cuda", generator=gen) < 0.01, -math.inf)
        s["cum"] = -2 * torch.rand(case["n_batch"], w, device="cuda", generator=gen) - 20
        s["finished"] = (torch.rand(case["n_batch"], w, device="cuda", generator=gen) < 0.1)
        s["eos"] = vocab // 2
        s["state"] = torch.randn(rows, case["segments"], case["positions"], case["dim"], device="cuda",
                                 generator=gen, dtype=torch.bfloat16)
        s["tokens"] = torch.zeros(case["n_batch"], w, dtype=torch.int32, device="cuda")
        s["parents"] = torch.zeros_like(s["tokens"])
        s["scores"] = torch.zeros(case["n_batch"], w, device="cuda")
        s["done"] = torch.zeros_like(s["finished"])
        if own:
            from persistent_megakernel_03_b200 import binding
            s["workspace"] = torch.empty(binding.beam_select_workspace_bytes(case["n_batch"], w, vocab),
                                         dtype=torch.uint8, device="cuda")
        return s
    lens, heads, dim, n_seq = _lens(case), case["kv_heads"], case["dim"], case["n_seq"]
    s["most"] = max(lens)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if case["kind"] == "prompt":
        s["page"], pages, s["table"] = _pages(gen, n_seq, s["most"], case["page"])
        s["pool"] = torch.zeros(pages, heads * s["page"] * (dim + dim // 8), dtype=torch.uint8, device="cuda")
        s["k"], s["v"] = _keys_values(gen, sum(lens), heads, dim, DTYPES[case["dtype"]])
        new = lens
        s["k_out"] = torch.zeros(n_seq, max(1, s["most"]), heads, dim, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
    else:
        s["page"], s["pool"], s["table"] = _filled(gen, case, lens)
        keys = s["table"].shape[1] * s["page"]
        # weight a key has gathered: a few have most of it, the newest have none yet
        s["weight"] = torch.exp(2 * torch.randn(n_seq, heads, keys, device="cuda", generator=gen) - 4)
        s["weight"].masked_fill_(torch.rand(n_seq, heads, keys, device="cuda", generator=gen) < 0.05, 0.0)
    if case["kind"] in ("attend", "step"):
        q_heads, q_len = heads * case["group"], case["q_len"]
        s["q"] = torch.randn(n_seq, q_len, q_heads, dim, device="cuda", generator=gen).to(DTYPES[case["dtype"]])
        s["out"] = torch.zeros_like(s["q"])
        if case["kind"] == "step":
            new = [min(n, q_len) for n in lens]
            s["k"], s["v"] = _keys_values(gen, sum(new), heads, dim, DTYPES[case["dtype"]])
    if case["kind"] == "evict":
        budget = case["budget"]
        s["dst_page"], pages, s["dst_table"] = _pages(gen, n_seq, budget, case["page"])
        s["dst_pool"] = torch.zeros(pages, heads * s["dst_page"] * (dim + dim // 8), dtype=torch.uint8, device="cuda")
        s["dst_weight"] = torch.zeros(n_seq, heads, s["dst_table"].shape[1] * s["dst_page"], device="cuda")
        s["dst_lens"] = s["lens"].clamp(max=budget)
        s["kept"] = torch.zeros(n_seq, heads, budget, dtype=torch.int32, device="cuda")
        s["k_out"] = torch.zeros(n_seq, budget, heads, dim, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
    if case["kind"] in ("prompt", "step"):
        s["offsets"] = torch.tensor([sum(new[:i]) for i in range(n_seq + 1)], dtype=torch.int32, device="cuda")
    if own:
        from persistent_megakernel_03_b200 import binding
        s["cache"] = binding.Kv4Cache(s["pool"], s["lens"], heads, dim, s["page"], s["table"], s.get("weight"))
        if case["kind"] == "evict":
            s["dst"] = binding.Kv4Cache(s["dst_pool"], s["dst_lens"], heads, dim, s["dst_page"], s["dst_table"],
                                        s["dst_weight"])
        if case["kind"] in ("attend", "step"):
            n = binding.attention_kv4_workspace_bytes(s["cache"], case["q_len"], heads * case["group"],
                                                      case["accumulate"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------- plain forms

def _append_plain(s):
    n = s["k"].shape[0]
    if n:
        at = torch.arange(n, device="cuda")
        seq = torch.searchsorted(s["offsets"][1:].contiguous().long(), at, right=True)
        slot = s["lens"].long()[seq] - s["offsets"].long()[seq + 1] + at
        _store(s["pool"], s["table"], s["page"], s["kv_heads"], s["dim"], seq, slot, s["k"], s["v"])
        if "weight" in s:   # a new key has gathered none
            s["weight"][seq, :, slot] = 0.0


def _attend_plain(s):
    n_seq, q_len, heads, dim = s["n_seq"], s["q_len"], s["kv_heads"], s["dim"]
    keys = max(1, s["most"])
    k, v = _values(s["pool"], s["table"], s["page"], heads, dim, keys)
    q = s["q"].float().view(n_seq, q_len, heads, -1, dim).permute(0, 2, 1, 3, 4)  # [n_seq][heads][q_len][group]
    x = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)) * dim ** -0.5
    j = torch.arange(keys, device="cuda")
    limit = s["lens"].view(-1, 1) - q_len + 1 + torch.arange(q_len, device="cuda")     # keys that a token sees
    seen = (j < limit.unsqueeze(-1)).repeat_interleave(s["group"], 1).unsqueeze(1)
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    out = torch.matmul(p, v).unflatten(2, (q_len, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s["out"].copy_(out)
    if s["accumulate"]:
        s["weight"][:, :, :keys] += p.sum(2)
        return {"out": s["out"], "weight": s["weight"]}
    return {"out": s["out"]}


def _read_plain(pool, table, page, heads, dim, lens, k_out, v_out):
    keys = k_out.shape[1]
    have = (torch.arange(keys, device="cuda") < lens.view(-1, 1)).view(-1, keys, 1, 1)
    for x, out in zip(_values(pool, table, page, heads, dim, keys), (k_out, v_out)):
        out.copy_(torch.where(have, x.transpose(1, 2), out.float()))
    return {"k": k_out, "v": v_out}


def _evict_plain(s):
    n_seq, heads, dim, budget = s["n_seq"], s["kv_heads"], s["dim"], s["budget"]
    keys = s["weight"].shape[2]
    j = torch.arange(keys, device="cuda")
    lens = s["lens"].long().view(-1, 1, 1)
    kept_always = (j < s["first"]) | (j >= lens - s["last"])
    rank = torch.where(kept_always, torch.full_like(s["weight"], math.inf), s["weight"])
    rank = torch.where(j < lens, rank, torch.full_like(rank, -math.inf))
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :budget]
    if keys < budget:
        order = torch.cat((order, torch.full((n_seq, heads, budget - keys), keys, device="cuda")), -1)
    live = torch.arange(budget, device="cuda") < lens.clamp(max=budget)
    order = torch.where(live, order, torch.full_like(order, keys)).sort(-1).values
    slot = order.clamp(max=keys - 1)
    s["kept"].copy_(torch.where(live, order, torch.full_like(order, -1)))
    live = live.expand(n_seq, heads, budget)
    seq, head, to = live.nonzero(as_tuple=True)
    src = slot[seq, head, to]
    s["dst_weight"][seq, head, to] = s["weight"][seq, head, src]
    here, there = _regions(s["pool"], heads, dim), _regions(s["dst_pool"], heads, dim)
    a = s["table"][seq, src // s["page"]].long(), head, src % s["page"] // BLOCK, src % BLOCK
    b = s["dst_table"][seq, to // s["dst_page"]].long(), head, to % s["dst_page"] // BLOCK, to % BLOCK
    there[0][b], there[1][b], there[2][b], there[3][b] = (x[a] for x in here)
    got = _read_plain(s["dst_pool"], s["dst_table"], s["dst_page"], heads, dim, s["dst_lens"], s["k_out"], s["v_out"])
    return {"kept": s["kept"], "weight": s["dst_weight"], **got}


def _beam_plain(s):
    n_batch, w, vocab = s["n_batch"], s["beams"], s["vocab"]
    # scores of different beams lie close together: 64 bits, as a border between them asks for
    x = s["logits"].double().view(n_batch, w, vocab)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    score = s["cum"].double().unsqueeze(-1) + (x - top) - torch.exp(x - top).sum(-1, keepdim=True).log()
    score = torch.where(torch.isnan(score), torch.full_like(score, -math.inf), score)
    only = torch.full_like(score, -math.inf)
    only[..., s["eos"]] = s["cum"].double()
    score = torch.where(s["finished"].unsqueeze(-1), only, score).flatten(1)
    # the highest w of each search, ties to the lowest place
    best, at = _first(score, w)
    dead = torch.isinf(best)
    me = torch.arange(w, device="cuda").expand(n_batch, w)
    parents = torch.where(dead, me, at // vocab)
    tokens = torch.where(dead, torch.full_like(at, s["eos"]), at % vocab)
    s["tokens"].copy_(tokens)
    s["parents"].copy_(parents)
    s["scores"].copy_(best)
    s["done"].copy_(s["finished"].gather(1, parents) | (tokens == s["eos"]))
    moved = s["state"][:, :, s["first"]:s["first"] + s["count"]]
    rows = (parents + torch.arange(n_batch, device="cuda").unsqueeze(1) * w).flatten()
    moved.copy_(moved[rows])
    return {"tokens": s["tokens"], "parents": s["parents"], "scores": s["scores"], "done": s["done"],
            "state": s["state"]}


def _first(score, w):
    """The w highest of each row and their places, equal ones by the lowest place."""
    border = torch.topk(score, w, -1).values[:, -1:]
    # all above the border, and of those on it the lowest places: a stable order of few values
    place = torch.where(score >= border, torch.arange(score.shape[1], device=score.device), score.shape[1])
    some = torch.where(score > border, place, score.shape[1])
    edge = torch.where(score == border, place, score.shape[1])
    at = torch.cat((torch.topk(some, w, -1, largest=False).values, torch.topk(edge, w, -1, largest=False).values), -1)
    value = torch.where(at < score.shape[1], score.gather(1, at.clamp(max=score.shape[1] - 1)),
                        torch.full_like(at, -math.inf, dtype=score.dtype))
    value = torch.where(at < score.shape[1], value, torch.full_like(value, -math.inf))
    order = torch.sort(value, dim=-1, descending=True, stable=True).indices[:, :w]
    return value.gather(1, order), at.gather(1, order)


# ---------------------------------------------------------------- one pass

def run(state):
    s, kind = state, state["kind"]
    if not own:
        if kind == "beam":
            return _beam_plain(s)
        if kind == "evict":
            return _evict_plain(s)
        if kind != "attend":
            _append_plain(s)
        if kind == "prompt":
            return _read_plain(s["pool"], s["table"], s["page"], s["kv_heads"], s["dim"], s["lens"], s["k_out"], s["v_out"])
        return _attend_plain(s)
    from persistent_megakernel_03_b200 import binding
    if kind == "beam":
        binding.beam_select(s["logits"], s["cum"], s["tokens"], s["parents"], s["scores"], s["workspace"],
                            finished=s["finished"], finished_out=s["done"], eos=s["eos"])
        binding.beam_reorder(s["state"], s["parents"], s["first"], s["count"])
        return {"tokens": s["tokens"], "parents": s["parents"], "scores": s["scores"], "done": s["done"],
                "state": s["state"]}
    if kind == "evict":
        binding.kv4_evict(s["cache"], s["dst"], s["budget"], s["first"], s["last"], s["kept"])
        binding.kv4_read(s["dst"], s["k_out"], s["v_out"])
        return {"kept": s["kept"], "weight": s["dst_weight"], "k": s["k_out"], "v": s["v_out"]}
    if kind != "attend":
        binding.kv4_append(s["cache"], s["k"], s["v"], s["offsets"])
    if kind == "prompt":
        binding.kv4_read(s["cache"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    binding.attention_kv4(s["cache"], s["q"], s["out"], s["workspace"], accumulate=s["accumulate"])
    return {"out": s["out"], "weight": s["weight"]} if s["accumulate"] else {"out": s["out"]}


# --------------------------------------------------------- 64 bits, by hand

def _row64(codes, scales):
    """Bytes of rows [n][dim / 2] and [n][dim / 16] as the numbers they stand for, from the formats' bits."""
    c = torch.stack((codes % 16, codes // 16), 2).reshape(codes.shape[0], -1).long()
    e, m = (c // 2) % 4, c % 2
    mag = torch.where(e == 0, m * 0.5, (1 + 0.5 * m) * 2.0 ** (e - 1).double())
    b = scales.long()
    big, small = (b // 8) % 16, b % 8
    s = torch.where(big == 0, small * 2.0 ** -9, (1 + small / 8.0) * 2.0 ** (big - 7).double())
    return torch.where(c >= 8, -mag, mag) * s.repeat_interleave(GROUP, 1)


def _head64(s, seq, head, n, pool="pool", table="table", page="page"):
    """K and V of slots [0, n) of one sequence and head, 64 bits."""
    dim, per = s["dim"], s[page]
    size, half, few = BLOCK * (s["dim"] + s["dim"] // 8), BLOCK * dim // 2, BLOCK * dim // GROUP
    raw = s[pool].view(s[pool].shape[0], s["kv_heads"], per // BLOCK, size)
    got = raw[s[table][seq].long(), head].reshape(-1, size)
    cut = [got[:, a:b].reshape(got.shape[0] * BLOCK, -1)[:n]
           for a, b in ((0, half), (half, half + few), (half + few, 2 * half + few), (2 * half + few, size))]
    return _row64(cut[0], cut[1]), _row64(cut[2], cut[3])


def _round64(x):
    """What the cache holds of rows x [n][dim]: the nearest scale and the nearest codes, by distance."""
    scale_of = torch.arange(127, device="cuda")
    grid = torch.where(scale_of < 8, scale_of * 2.0 ** -9, (1 + (scale_of % 8) / 8.0) * 2.0 ** (scale_of // 8 - 7).double())
    mags = torch.tensor(E2M1, dtype=torch.float64, device="cuda")

    def nearest(y, values):
        up = torch.searchsorted(values, y).clamp(1, len(values) - 1)
        low = up - 1
        a, b = (y - values[low]).abs(), (values[up] - y).abs()
        return torch.where((b < a) | ((b == a) & (up % 2 == 0)), up, low)

    g = x.double().reshape(x.shape[0], -1, GROUP)
    s = grid[nearest((g.abs().amax(2) / 6).clamp(max=448), grid)].unsqueeze(2)
    y = torch.where(s > 0, g.abs() / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(g))
    return (torch.sign(g) * mags[nearest(y.clamp(max=6), mags)] * s).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "beam":
        return _beam64(s)
    lens, heads, dim = _lens(case), case["kv_heads"], case["dim"]
    if case["kind"] == "prompt":
        out = [torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
        for i, n in enumerate(lens):
            a = sum(lens[:i])
            for x, to in zip((s["k"], s["v"]), out):
                for h in range(heads):
                    to[i, :n, h] = _round64(x[a:a + n, h]) if n else 0
        return {"k": out[0], "v": out[1]}
    if case["kind"] == "evict":
        return _evict64(s, lens)
    q_len, group = case["q_len"], case["group"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    weight = s["weight"].double()
    for i, n in enumerate(lens):
        for h in range(heads):
            if n == 0:
                continue
            k, v = _head64(s, i, h, n)
            if case["kind"] == "step":
                new, a = min(n, q_len), int(s["offsets"][i])
                k[n - new:] = _round64(s["k"][a:a + new, h])
                v[n - new:] = _round64(s["v"][a:a + new, h])
                weight[i, h, n - new:n] = 0
            for t in range(q_len):
                see = n - q_len + t + 1
                if see > 0:
                    q = s["q"][i, t, h * group:(h + 1) * group].double()
                    p = torch.softmax(q @ k[:see].T / math.sqrt(dim), 1)
                    out[i, t, h * group:(h + 1) * group] = p @ v[:see]
                    weight[i, h, :see] += p.sum(0)
    return {"out": out, "weight": weight} if case["accumulate"] else {"out": out}


def _evict64(s, lens):
    heads, budget = s["kv_heads"], s["budget"]
    kept = torch.full(s["kept"].shape, -1, dtype=torch.int64, device="cuda")
    weight = torch.zeros(s["dst_weight"].shape, dtype=torch.float64, device="cuda")
    k_out = torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda")
    v_out = torch.zeros_like(k_out)
    for i, n in enumerate(lens):
        for h in range(heads):
            if n == 0:
                continue
            w = s["weight"][i, h, :n].double()
            if n <= budget:
                at = torch.arange(n, device="cuda")
            else:
                sure = torch.zeros(n, dtype=torch.bool, device="cuda")
                sure[:s["first"]] = True
                sure[n - s["last"]:] = True
                rest = (~sure).nonzero().flatten()
                take = budget - int(sure.sum())
                pick = rest[torch.sort(-w[rest], stable=True).indices[:take]]
                at = torch.cat((sure.nonzero().flatten(), pick)).sort().values
            m = len(at)
            kept[i, h, :m] = at
            weight[i, h, :m] = w[at]
            k, v = _head64(s, i, h, n)
            k_out[i, :m, h], v_out[i, :m, h] = k[at], v[at]
    return {"kept": kept, "weight": weight, "k": k_out, "v": v_out}


def _beam64(s):
    n_batch, w, vocab, eos = s["n_batch"], s["beams"], s["vocab"], s["eos"]
    tokens, parents, scores, done = [], [], [], []
    for b in range(n_batch):
        found = []
        for i in range(w):
            cum = float(s["cum"][b, i])
            if bool(s["finished"][b, i]):
                found.append((-cum, i, eos))
                continue
            x = s["logits"][b * w + i].double()
            best = torch.sort(x, descending=True, stable=True)
            lse = float(torch.logsumexp(x, 0))
            found += [(-(cum + float(v) - lse), i, int(t)) for v, t in zip(best.values[:w], best.indices[:w])
                      if float(v) > -math.inf]
        found = sorted(found)[:w]
        found += [(math.inf, i, eos) for i in range(len(found), w)]
        tokens.append([t for _, _, t in found])
        parents.append([i for _, i, _ in found])
        scores.append([-x for x, _, _ in found])
        done.append([bool(s["finished"][b, i]) or t == eos for _, i, t in found])
    at = torch.tensor(parents, device="cuda")
    rows = (at + torch.arange(n_batch, device="cuda").view(-1, 1) * w).flatten()
    state = s["state"].double()
    part = slice(s["first"], s["first"] + s["count"])
    state[:, :, part] = state[rows][:, :, part]
    return {"tokens": torch.tensor(tokens, device="cuda"), "parents": at,
            "scores": torch.tensor(scores, dtype=torch.float64, device="cuda"),
            "done": torch.tensor(done, device="cuda"), "state": state}
