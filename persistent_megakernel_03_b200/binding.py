"""ctypes binding of libmk (include/mk.h): argument marshalling only.

Every step of the decode path runs in libmk's CUDA kernels; this module only
converts Python / torch arguments to the C-ABI's plain pointers and sizes.
torch provides device memory and streams.  When libmk.so cannot be loaded the
binding raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Dict, List, Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
# MK_LIBRARY selects another build of the library (A/B comparisons of builds).
LIB_PATH = os.environ.get("MK_LIBRARY") or os.path.join(HERE, "libmk.so")

MK_OK = 0
ERRORS = {-1: "MK_ERR_INVALID_ARG", -2: "MK_ERR_OOM", -3: "MK_ERR_CUDA", -4: "MK_ERR_TIMEOUT",
          -5: "MK_ERR_POS_RANGE", -6: "MK_ERR_NOT_RESIDENT", -7: "MK_ERR_POISONED",
          -8: "MK_ERR_TOKEN_RANGE", -9: "MK_ERR_UNSUPPORTED", -10: "MK_ERR_BOUNDS"}
MODE_MEGAKERNEL, MODE_PER_OP, MODE_PER_OP_GRAPH = 0, 1, 2
ACT_Q, ACT_ATTN, ACT_FFN, ACT_X = 0, 1, 2, 3
TASK_KINDS = ("QKV", "ATTN", "OPROJ", "GATEUP", "DOWN", "LMHEAD")

EXPORTS = ("mk_create", "mk_prefill", "mk_decode_step", "mk_decode_steps", "mk_decode_step_host",
           "mk_copy_hidden", "mk_copy_activation", "mk_prefill_slots", "mk_decode_step_slots",
           "mk_kv_release", "mk_kv_set_pages", "mk_kv_get_pages", "mk_kv_free_pages",
           "mk_build_flags",
           "mk_kv_pointer", "mk_copy_kv", "mk_set_mode", "mk_status", "mk_last_error",
           "mk_destroy", "mk_plan_build", "mk_plan_get_info", "mk_plan_get_tasks",
           "mk_plan_get_queue", "mk_plan_get_event_counts", "mk_plan_destroy",
           "mk_qkv_row_source", "mk_read_probe", "mk_set_trace", "mk_set_prefill_trace", "mk_inject_prefill_stall", "mk_prefill_graph",
           "mk_prefill_layout",
           "mk_attention_workspace_bytes", "mk_attention_decode",
           "mk_attention_decode_noalloc", "mk_inject_stall", "mk_kv_reorder",
           "mk_kv4_page_bytes", "mk_kv4_append", "mk_kv4_read", "mk_kv4_evict", "mk_kv4_reorder",
           "mk_attention_kv4_workspace_bytes", "mk_attention_kv4", "mk_beam_select_workspace_bytes",
           "mk_beam_select", "mk_beam_reorder")


class MkError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{ERRORS.get(code, code)}: {msg}")
        self.code = code


class Config(C.Structure):
    _fields_ = [("n_layers", C.c_int), ("hidden", C.c_int), ("n_q_heads", C.c_int),
                ("n_kv_heads", C.c_int), ("head_dim", C.c_int), ("ffn", C.c_int),
                ("vocab", C.c_int), ("rms_eps", C.c_float), ("rope_theta", C.c_double),
                ("qkv_bias", C.c_int), ("tied_embeddings", C.c_int), ("max_seq", C.c_int),
                ("max_batch", C.c_int)]


LAYER_FIELDS = ("attn_norm", "wq", "wk", "wv", "bq", "bk", "bv", "wo", "ffn_norm", "w_gate",
                "w_up", "w_down")


class LayerWeights(C.Structure):
    _fields_ = [(k, C.c_void_p) for k in LAYER_FIELDS]


class Weights(C.Structure):
    _fields_ = [("embed", C.c_void_p), ("layers", C.POINTER(LayerWeights)),
                ("final_norm", C.c_void_p), ("lm_head", C.c_void_p)]


class Options(C.Structure):
    _fields_ = [("num_ctas", C.c_int), ("attn_splits", C.c_int), ("timeout_ms", C.c_int),
                ("mode", C.c_int), ("l2_prefetch", C.c_int), ("weight_format", C.c_int),
                ("batch_sequential", C.c_int), ("prefill_steps", C.c_int),
                ("kv_page_tokens", C.c_int), ("kv_pool_pages", C.c_int),
                ("prefill_per_operator", C.c_int), ("prefill_attention", C.c_int)]


class Kv4Struct(C.Structure):
    _fields_ = [("n_kv_heads", C.c_int), ("head_dim", C.c_int), ("page_tokens", C.c_int),
                ("n_pages", C.c_int), ("n_seq", C.c_int), ("pages_per_seq", C.c_int),
                ("k_log2", C.c_int), ("v_log2", C.c_int), ("pool_dev", C.c_void_p),
                ("table_dev", C.c_void_p), ("lens_dev", C.c_void_p), ("scores_dev", C.c_void_p)]


class PlanInfo(C.Structure):
    _fields_ = [("num_ctas", C.c_int), ("n_tasks", C.c_int), ("n_events", C.c_int),
                ("n_stages", C.c_int), ("attn_splits", C.c_int), ("n_lm_tasks", C.c_int),
                ("ring_slots", C.c_int), ("slot_bytes", C.c_int), ("smem_bytes", C.c_int),
                ("threads_per_cta", C.c_int), ("weight_bytes_per_step", C.c_longlong)]


class PlanTask(C.Structure):
    _fields_ = [("kind", C.c_int), ("layer", C.c_int), ("row0", C.c_int), ("row1", C.c_int),
                ("req", C.c_int), ("wait_event", C.c_int), ("wait_count", C.c_int),
                ("signal_event0", C.c_int), ("n_signal", C.c_int), ("cta", C.c_int),
                ("stage", C.c_int)]


_lib = None


def lib(build_if_missing: bool = True):
    """Loads libmk.so (building it with nvcc when absent); raises on failure."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH) and build_if_missing and not os.environ.get("MK_LIBRARY"):
        from . import build as _build
        _build.build()
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libmk.so not found at {LIB_PATH}; run the package build")
    L = C.CDLL(LIB_PATH)
    vp, ip, i = C.c_void_p, C.POINTER(C.c_int32), C.c_int
    L.mk_create.argtypes = [C.POINTER(Config), C.POINTER(Weights), C.POINTER(Options), vp,
                            C.POINTER(vp)]
    L.mk_prefill.argtypes = [vp, vp, ip, i, vp, vp]
    L.mk_decode_step.argtypes = [vp, vp, ip, i, vp, vp]
    L.mk_decode_step_host.argtypes = [vp, ip, ip, i, ip]
    L.mk_decode_steps.argtypes = [vp, vp, i, i, vp, vp]
    L.mk_copy_hidden.argtypes = [vp, vp, i]
    L.mk_copy_activation.argtypes = [vp, i, vp, i]
    L.mk_prefill_slots.argtypes = [vp, vp, ip, ip, i, vp, vp]
    L.mk_decode_step_slots.argtypes = [vp, vp, ip, ip, i, vp, vp]
    L.mk_kv_release.argtypes = [vp, i]
    L.mk_kv_set_pages.argtypes = [vp, i, ip, i]
    L.mk_kv_get_pages.argtypes = [vp, i, ip, i]
    L.mk_kv_free_pages.argtypes = [vp]
    L.mk_build_flags.argtypes = []
    L.mk_build_flags.restype = i
    L.mk_kv_pointer.argtypes = [vp, i, i, i, i, C.POINTER(vp)]
    L.mk_copy_kv.argtypes = [vp, i, i, i, i, i, vp]
    L.mk_set_mode.argtypes = [vp, i]
    L.mk_status.argtypes = [vp]
    L.mk_last_error.argtypes = [vp]
    L.mk_last_error.restype = C.c_char_p
    L.mk_destroy.argtypes = [vp]
    L.mk_destroy.restype = None
    L.mk_inject_stall.argtypes = [vp, i]
    L.mk_inject_prefill_stall.argtypes = [vp, i]
    L.mk_prefill_graph.argtypes = [vp, i, vp, i, vp, i, vp, i, vp, vp, i, vp, vp]
    L.mk_prefill_layout.argtypes = [vp, vp, i, i, vp, i, vp, i, vp, vp, vp]
    L.mk_plan_build.argtypes = [C.POINTER(Config), C.POINTER(Options), i, C.POINTER(vp)]
    L.mk_plan_get_info.argtypes = [vp, C.POINTER(PlanInfo)]
    L.mk_plan_get_tasks.argtypes = [vp, C.POINTER(PlanTask), i]
    L.mk_plan_get_queue.argtypes = [vp, i, ip, i]
    L.mk_plan_get_event_counts.argtypes = [vp, ip, i]
    L.mk_plan_destroy.argtypes = [vp]
    L.mk_plan_destroy.restype = None
    L.mk_qkv_row_source.argtypes = [C.POINTER(Config), i, ip, ip, ip]
    L.mk_read_probe.argtypes = [vp, C.c_size_t, vp, vp]
    L.mk_set_trace.argtypes = [vp, vp]
    L.mk_set_prefill_trace.argtypes = [vp, vp, C.c_int]
    L.mk_attention_workspace_bytes.argtypes = [i, i, i]
    L.mk_attention_workspace_bytes.restype = C.c_size_t
    L.mk_attention_decode.argtypes = [vp, vp, vp, i, i, i, i, vp, vp, vp]
    L.mk_attention_decode_noalloc.argtypes = [vp, vp, vp, i, i, i, i, vp, vp]
    ll, sz, f = C.c_longlong, C.c_size_t, C.c_float
    L.mk_kv_reorder.argtypes = [vp, ip, i, vp, i, i]
    L.mk_kv4_page_bytes.argtypes = [i, i, i]
    L.mk_kv4_page_bytes.restype = sz
    L.mk_kv4_append.argtypes = [vp, vp, vp, i, ll, ll, vp, i, vp]
    L.mk_kv4_read.argtypes = [vp, i, i, vp, vp, vp]
    L.mk_kv4_evict.argtypes = [vp, vp, i, i, i, vp, vp]
    L.mk_kv4_reorder.argtypes = [vp, vp, i, i, i, vp]
    L.mk_attention_kv4_workspace_bytes.argtypes = [vp, i, i, i]
    L.mk_attention_kv4_workspace_bytes.restype = sz
    L.mk_attention_kv4.argtypes = [vp, vp, i, i, i, ll, f, i, vp, sz, vp, vp]
    L.mk_beam_select_workspace_bytes.argtypes = [i, i, i]
    L.mk_beam_select_workspace_bytes.restype = sz
    L.mk_beam_select.argtypes = [vp, i, ll, vp, vp, i, i, i, i, vp, vp, vp, vp, vp, sz, vp]
    L.mk_beam_reorder.argtypes = [vp, vp, i, i, sz, i, sz, sz, vp]
    _lib = L
    return L


def make_config(model, max_seq: int, max_batch: int = 1) -> Config:
    return Config(model.n_layers, model.hidden, model.n_q_heads, model.n_kv_heads,
                  model.head_dim, model.ffn, model.vocab, float(model.rms_eps),
                  float(model.rope_theta), int(bool(model.qkv_bias)),
                  int(bool(model.tied_embeddings)), int(max_seq), int(max_batch))


def _ints(vals: Sequence[int]):
    return (C.c_int32 * len(vals))(*[int(v) for v in vals])


def _check(rc: int, h=None):
    if rc != MK_OK:
        msg = lib().mk_last_error(h).decode(errors="replace")
        raise MkError(rc, msg)


# ------------------------------------------------------------------ plan

def prefill_layout(offsets, slots, max_tokens: int):
    """How mk_prefill lays out a call's positions for the persistent prefill
    (host only, see mk_prefill_layout): (positions as rows of (token index,
    slot, position, request or -1), attention runs as rows of (block, first
    block position, count, slot, first position), folded flag per request)."""
    L = lib()
    n_req = len(offsets) - 1
    off_c = (C.c_int32 * len(offsets))(*[int(v) for v in offsets])
    sl_c = (C.c_int32 * n_req)(*[int(v) for v in slots])
    n_pos, n_runs = C.c_int(0), C.c_int(0)
    rc = L.mk_prefill_layout(off_c, sl_c, n_req, max_tokens, None, 0, None, 0, C.byref(n_pos),
                             C.byref(n_runs), None)
    if rc != MK_OK:
        raise MkError(rc, "mk_prefill_layout rejected the call")
    pos_c = (C.c_int32 * (4 * n_pos.value))()
    runs_c = (C.c_int32 * (5 * n_runs.value))()
    fold_c = (C.c_int32 * n_req)()
    _check(L.mk_prefill_layout(off_c, sl_c, n_req, max_tokens, pos_c, n_pos.value, runs_c,
                               n_runs.value, C.byref(n_pos), C.byref(n_runs), fold_c))
    positions = [tuple(pos_c[4 * t:4 * t + 4]) for t in range(n_pos.value)]
    runs = [tuple(runs_c[5 * i:5 * i + 5]) for i in range(n_runs.value)]
    return positions, runs, [bool(v) for v in fold_c]


def prefill_graph(model, T: int, tiles, lm_req, num_ctas: int):
    """The persistent prefill's task graph of one block (host only, see
    mk_prefill_graph): (tasks as rows of 9 ints, queue offsets, queues, number
    of events)."""
    L = lib()
    cfg = make_config(model, max(T, 1), 1)
    flat = [int(v) for t in tiles for v in t]
    tiles_c = (C.c_int32 * len(flat))(*flat)
    lm_c = (C.c_int32 * T)(*[int(v) for v in lm_req])
    n_tasks, n_events = C.c_int(0), C.c_int(0)
    rc = L.mk_prefill_graph(C.byref(cfg), T, tiles_c, len(tiles), lm_c, num_ctas, None, 0, None,
                            None, 0, C.byref(n_tasks), C.byref(n_events))
    if rc != MK_OK:
        raise MkError(rc, "mk_prefill_graph rejected the block")
    n = n_tasks.value
    tasks = (C.c_int32 * (9 * n))()
    qoff = (C.c_int32 * (num_ctas + 1))()
    queue = (C.c_int32 * n)()
    _check(L.mk_prefill_graph(C.byref(cfg), T, tiles_c, len(tiles), lm_c, num_ctas, tasks, n, qoff,
                              queue, n, C.byref(n_tasks), C.byref(n_events)))
    rows = [list(tasks[9 * i:9 * i + 9]) for i in range(n)]
    return rows, list(qoff), list(queue), n_events.value


class Plan:
    """The task graph mk_create would build (host only)."""

    def __init__(self, model, max_seq: int, num_ctas: int, max_batch: int = 1,
                 attn_splits: int = 0, weight_format: int = 0):
        L = lib()
        self.h = C.c_void_p()
        cfg = make_config(model, max_seq, max_batch)
        opt = Options(num_ctas, attn_splits, 0, 0, 0, weight_format, 0, 0, 0, 0, 0, 0)
        rc = L.mk_plan_build(C.byref(cfg), C.byref(opt), int(num_ctas), C.byref(self.h))
        if rc != MK_OK:
            raise MkError(rc, "mk_plan_build rejected the configuration")
        self.info = PlanInfo()
        _check(L.mk_plan_get_info(self.h, C.byref(self.info)))

    def tasks(self) -> List[dict]:
        n = self.info.n_tasks
        arr = (PlanTask * n)()
        got = lib().mk_plan_get_tasks(self.h, arr, n)
        assert got == n
        return [{f: getattr(t, f) for f, _ in PlanTask._fields_} for t in arr]

    def queue(self, cta: int) -> List[int]:
        n = lib().mk_plan_get_queue(self.h, cta, None, 0)
        buf = (C.c_int32 * max(n, 1))()
        lib().mk_plan_get_queue(self.h, cta, buf, n)
        return list(buf[:n])

    def event_counts(self) -> List[int]:
        n = lib().mk_plan_get_event_counts(self.h, None, 0)
        buf = (C.c_int32 * max(n, 1))()
        lib().mk_plan_get_event_counts(self.h, buf, n)
        return list(buf[:n])

    def __del__(self):
        if getattr(self, "h", None):
            lib().mk_plan_destroy(self.h)
            self.h = None


def qkv_row_source(model, r: int):
    cfg = make_config(model, 1)
    w, h, d = C.c_int32(), C.c_int32(), C.c_int32()
    _check(lib().mk_qkv_row_source(C.byref(cfg), int(r), C.byref(w), C.byref(h), C.byref(d)))
    return w.value, h.value, d.value


# ---------------------------------------------------------------- decoder

class Decoder:
    """One libmk context.  ``weights`` maps the synthetic generator's names to
    CUDA bf16 tensors; mk_create copies them, so they may be dropped after."""

    def __init__(self, model, weights: Dict[str, "torch.Tensor"], max_seq: int,
                 max_batch: int = 1, num_ctas: int = 0, attn_splits: int = 0,
                 timeout_ms: int = 0, mode: int = MODE_MEGAKERNEL, stream=None,
                 l2_prefetch: int = 0, prefill_steps: int = 0, batch_sequential: int = 0,
                 weight_format: int = 0, kv_page_tokens: int = 0, kv_pool_pages: int = 0,
                 prefill_per_operator: int = 0, prefill_attention: int = 0):
        import torch
        L = lib()
        self.model = model
        self.max_seq = max_seq
        self.max_batch = max_batch
        self.stream = stream if stream is not None else torch.cuda.current_stream()

        def ptr(name):
            t = weights.get(name)
            if t is None:
                return None
            assert t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous(), name
            return t.data_ptr()

        layers = (LayerWeights * model.n_layers)()
        for l in range(model.n_layers):
            for k in LAYER_FIELDS:
                setattr(layers[l], k, ptr(f"layers.{l}.{k}"))
        w = Weights(ptr("embed"), layers, ptr("final_norm"),
                    None if model.tied_embeddings else ptr("lm_head"))
        cfg = make_config(model, max_seq, max_batch)
        opt = Options(num_ctas, attn_splits, timeout_ms, mode, l2_prefetch, weight_format,
                      batch_sequential, prefill_steps, kv_page_tokens, kv_pool_pages,
                      prefill_per_operator, prefill_attention)
        self.h = C.c_void_p()
        rc = L.mk_create(C.byref(cfg), C.byref(w), C.byref(opt), self.stream.cuda_stream,
                         C.byref(self.h))
        if rc != MK_OK:
            msg = L.mk_last_error(None).decode(errors="replace")
            self.h = None
            raise MkError(rc, msg)

    def close(self):
        if getattr(self, "h", None):
            lib().mk_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # interpreter shutdown: the library may be gone already
            pass

    def set_mode(self, mode: int):
        _check(lib().mk_set_mode(self.h, int(mode)), self.h)

    def prefill(self, tokens_dev, offsets: Sequence[int], logits_dev=None, next_ids_dev=None):
        n_req = len(offsets) - 1
        _check(lib().mk_prefill(self.h, tokens_dev.data_ptr(), _ints(offsets), n_req,
                                None if logits_dev is None else logits_dev.data_ptr(),
                                None if next_ids_dev is None else next_ids_dev.data_ptr()),
               self.h)

    def decode(self, tokens_dev, pos: Sequence[int], logits_dev=None, next_ids_dev=None):
        _check(lib().mk_decode_step(self.h, tokens_dev.data_ptr(), _ints(pos), len(pos),
                                    None if logits_dev is None else logits_dev.data_ptr(),
                                    None if next_ids_dev is None else next_ids_dev.data_ptr()),
               self.h)

    def prefill_slots(self, tokens_dev, offsets: Sequence[int], slots: Sequence[int],
                      logits_dev=None, next_ids_dev=None):
        """mk_prefill with request r on KV-cache slot slots[r]."""
        _check(lib().mk_prefill_slots(self.h, tokens_dev.data_ptr(), _ints(offsets), _ints(slots),
                                      len(slots),
                                      None if logits_dev is None else logits_dev.data_ptr(),
                                      None if next_ids_dev is None else next_ids_dev.data_ptr()),
               self.h)

    def decode_slots(self, tokens_dev, pos: Sequence[int], slots: Sequence[int], logits_dev=None,
                     next_ids_dev=None):
        """mk_decode_step with request r on KV-cache slot slots[r]."""
        _check(lib().mk_decode_step_slots(self.h, tokens_dev.data_ptr(), _ints(pos), _ints(slots),
                                          len(pos),
                                          None if logits_dev is None else logits_dev.data_ptr(),
                                          None if next_ids_dev is None else next_ids_dev.data_ptr()),
               self.h)

    def kv_release(self, slot: int):
        _check(lib().mk_kv_release(self.h, int(slot)), self.h)

    def kv_set_pages(self, slot: int, pages: Sequence[int]):
        _check(lib().mk_kv_set_pages(self.h, int(slot), _ints(pages), len(pages)), self.h)

    def kv_pages(self, slot: int) -> List[int]:
        n = lib().mk_kv_get_pages(self.h, int(slot), None, 0)
        _check(min(n, 0), self.h)
        out = (C.c_int32 * max(n, 1))()
        lib().mk_kv_get_pages(self.h, int(slot), out, n)
        return list(out)[:n]

    def kv_reorder(self, parents_dev, first: int, n_pos: int, slots: Optional[Sequence[int]] = None):
        """Positions [first, n_pos) of slot slots[b] (slot b without ``slots``)
        become those of slot slots[parents_dev[b]], in place (see
        mk_kv_reorder); ``parents_dev`` int32 CUDA, one entry per slot."""
        import torch
        _tensor(parents_dev, torch.int32, "parents_dev")
        n = parents_dev.numel() if slots is None else len(slots)
        if n != parents_dev.numel():
            raise ValueError("one parent per slot")
        _check(lib().mk_kv_reorder(self.h, None if slots is None else _ints(slots), n,
                                   parents_dev.data_ptr(), int(first), int(n_pos)), self.h)

    def beam_search(self, prompt_dev, beams: int, n_steps: int, eos: int = -1):
        """The ``beams`` best continuations of a prompt (int32 CUDA) of at most
        ``n_steps`` tokens, best first: (tokens [beams, n_steps] int32, sums of
        log-probabilities [beams] fp32).  Sequences that reached ``eos`` (>= 0)
        go on with it.  Uses slots 0..beams-1; after the prefill, steps,
        selection and the caches' reordering are enqueued without a host round
        trip on the decoder's stream, which waits for the caller's current
        stream first; that waits for the results."""
        import torch
        _tensor(prompt_dev, torch.int32, "prompt_dev")
        if not 1 <= beams <= self.max_batch:
            raise ValueError("beams is 1 to max_batch")
        n, V, dev = prompt_dev.numel(), self.model.vocab, prompt_dev.device
        if n_steps < 1 or n + n_steps - 1 > self.max_seq:
            raise ValueError("prompt and steps fit max_seq")
        caller = torch.cuda.current_stream(dev)
        apart = caller != self.stream
        if apart:      # the prompt may still be on its way
            self.stream.wait_stream(caller)
            prompt_dev.record_stream(self.stream)
        with torch.cuda.device(dev), torch.cuda.stream(self.stream):
            logits = torch.empty(beams, V, device=dev)
            cum, done = torch.full((2, 1, beams), float("-inf"), device=dev), None
            cum[0, 0, 0] = 0.0                # one live beam: the prompt's
            if eos >= 0:
                done = torch.zeros(2, 1, beams, dtype=torch.bool, device=dev)
            tok, par = torch.empty(2, 1, beams, dtype=torch.int32, device=dev)
            ws = torch.empty(beam_select_workspace_bytes(1, beams, V), dtype=torch.uint8, device=dev)
            seq = torch.empty(beams, n_steps, dtype=torch.int32, device=dev)
            self.prefill_slots(prompt_dev, [0, n], [0], logits[:1])
            logits[1:] = logits[:1]           # not read for candidates: their sums are -inf
            self.kv_reorder(torch.zeros(beams, dtype=torch.int32, device=dev), 0, n)
            for s in range(n_steps):
                a, b = s % 2, (s + 1) % 2
                beam_select(logits, cum[a], tok, par, cum[b], ws,
                            finished=None if done is None else done[a],
                            finished_out=None if done is None else done[b], eos=eos,
                            stream=self.stream)
                if s:
                    self.kv_reorder(par.view(-1), n, n + s)
                    seq[:, :s] = seq[:, :s][par.view(-1).long()]
                seq[:, s] = tok.view(-1)
                if s + 1 < n_steps:
                    self.decode_slots(tok.view(-1), [n + s] * beams, list(range(beams)), logits)
        sums = cum[n_steps % 2].view(-1)
        if apart:
            caller.wait_stream(self.stream)
            for t in (seq, sums):
                t.record_stream(caller)
        return seq, sums

    def kv_free_pages(self) -> int:
        n = lib().mk_kv_free_pages(self.h)
        _check(min(n, 0), self.h)
        return int(n)

    def decode_steps(self, token_dev, pos0: int, n_steps: int, ids_dev, last_logits_dev=None):
        """n_steps greedy steps in one persistent launch; ids_dev[s] gets step s's id."""
        _check(lib().mk_decode_steps(self.h, token_dev.data_ptr(), int(pos0), int(n_steps),
                                     ids_dev.data_ptr(),
                                     None if last_logits_dev is None else last_logits_dev.data_ptr()),
               self.h)

    def decode_host(self, tokens: Sequence[int], pos: Sequence[int]) -> List[int]:
        out = (C.c_int32 * len(tokens))()
        _check(lib().mk_decode_step_host(self.h, _ints(tokens), _ints(pos), len(tokens), out),
               self.h)
        return list(out)

    def copy_hidden(self, dst_dev, n_req: int = 1):
        _check(lib().mk_copy_hidden(self.h, dst_dev.data_ptr(), int(n_req)), self.h)

    def copy_activation(self, which: int, dst_dev):
        """The last single-request step's ACT_Q / ACT_ATTN / ACT_FFN / ACT_X vector
        (see mk_copy_activation) into the fp32 CUDA tensor ``dst_dev``."""
        _check(lib().mk_copy_activation(self.h, int(which), dst_dev.data_ptr(),
                                        int(dst_dev.numel())), self.h)

    def copy_kv(self, req: int, layer: int, kv_head: int, which: int, n: int, dst_dev):
        _check(lib().mk_copy_kv(self.h, req, layer, kv_head, which, n, dst_dev.data_ptr()),
               self.h)

    def set_trace(self, trace_dev=None):
        """Per-task timeline of later megakernel steps into ``trace_dev``
        (int64 CUDA tensor, 8 words per task); None turns it off."""
        _check(lib().mk_set_trace(self.h, None if trace_dev is None else trace_dev.data_ptr()),
               self.h)

    def set_prefill_trace(self, trace_dev=None):
        """Per-task timeline of the persistent prefill's first block into
        ``trace_dev`` (int64 CUDA tensor, 4 words per task); None turns it off."""
        cap = 0 if trace_dev is None else trace_dev.numel() // 4
        _check(lib().mk_set_prefill_trace(self.h, None if trace_dev is None else trace_dev.data_ptr(),
                                          cap), self.h)

    def status(self) -> int:
        return int(lib().mk_status(self.h))

    def inject_stall(self, task: int = -1):
        """Makes one task's event wait unreachable (failure-detection test hook):
        the next megakernel step ends with MK_ERR_TIMEOUT after timeout_ms."""
        _check(lib().mk_inject_stall(self.h, int(task)), self.h)

    def inject_prefill_stall(self, task: int = -1):
        """The same for the persistent prefill: the next prefill call ends with
        MK_ERR_TIMEOUT after 2 x timeout_ms."""
        _check(lib().mk_inject_prefill_stall(self.h, int(task)), self.h)

    def last_error(self) -> str:
        return lib().mk_last_error(self.h).decode(errors="replace")


def read_probe(src_dev, sink_dev, stream=None):
    """Enqueues one read-only pass over ``src_dev`` (a contiguous CUDA tensor)."""
    import torch
    st = stream if stream is not None else torch.cuda.current_stream()
    nbytes = src_dev.numel() * src_dev.element_size()
    _check(lib().mk_read_probe(src_dev.data_ptr(), nbytes, sink_dev.data_ptr(), st.cuda_stream))


def attention_workspace_bytes(n_q_per_kv: int, head_dim: int, splits: int) -> int:
    return int(lib().mk_attention_workspace_bytes(n_q_per_kv, head_dim, splits))


def attention_decode(q_dev, k_dev, v_dev, n_keys: int, splits: int, workspace_dev, out_dev,
                     stream=None):
    """Split-KV decode attention for one KV head (see mk_attention_decode)."""
    import torch
    st = stream if stream is not None else torch.cuda.current_stream()
    G, d = q_dev.shape
    _check(lib().mk_attention_decode(q_dev.data_ptr(), k_dev.data_ptr(), v_dev.data_ptr(),
                                     int(n_keys), int(G), int(d), int(splits),
                                     workspace_dev.data_ptr(), out_dev.data_ptr(), st.cuda_stream))


def attention_decode_noalloc(q_dev, k_dev, v_dev, n_keys: int, splits: int, out_dev,
                             stream=None):
    """mk_attention_decode with the library's static scratch instead of a
    caller workspace (see mk_attention_decode_noalloc)."""
    import torch
    st = stream if stream is not None else torch.cuda.current_stream()
    G, d = q_dev.shape
    _check(lib().mk_attention_decode_noalloc(q_dev.data_ptr(), k_dev.data_ptr(),
                                             v_dev.data_ptr(), int(n_keys), int(G), int(d),
                                             int(splits), out_dev.data_ptr(), st.cuda_stream))


# ------------------------------------- the state of a decode: 4-bit cache, beams

_DTYPES = {}   # MK_DTYPE_* by torch type, filled at the first use: this module loads without torch


def _dtype(t) -> int:
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"fp32, bf16 or fp16 expected, got {t.dtype}")
    return code


def _tensor(t, dtype, what, shape=None, device=None):
    """Pointer of a contiguous CUDA tensor, its type, shape and device (index) checked."""
    d = t.get_device()
    if d < 0 or (dtype is not None and t.dtype != dtype) or not t.is_contiguous():
        raise TypeError(f"{what}: a contiguous CUDA tensor{'' if dtype is None else f' of {dtype}'} expected")
    if device is not None and d != device:
        raise ValueError(f"{what}: on device {d}, the others on {device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(shape)} expected, got {tuple(t.shape)}")
    return t.data_ptr()


def _on(device, stream, call, *args):
    """Runs ``call(*args, stream)`` with the tensors' device (index) current; the
    stream is ``stream``, or that device's current one."""
    import torch
    raw = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
    if device == torch._C._cuda_getDevice():
        rc = call(*args, raw)
    else:
        with torch.cuda.device(device):
            rc = call(*args, raw)
    if rc:
        _check(rc)


def kv4_page_bytes(n_kv_heads: int, head_dim: int, page_tokens: int) -> int:
    return int(lib().mk_kv4_page_bytes(n_kv_heads, head_dim, page_tokens))


class Kv4Cache:
    """A 4-bit KV cache in the caller's tensors (see mk_kv4_cache): ``pool``
    uint8 [pages, kv4_page_bytes(...)], ``lens`` int32 [n_seq], ``table`` int32
    [n_seq, pages_per_seq] (None: sequence s owns the s-th run of pages),
    ``scores`` fp32 [n_seq, n_kv_heads, pages_per_seq * page_tokens] or None.
    Holds the tensors, copies nothing; their contents may change between
    calls, their storage not."""

    def __init__(self, pool, lens, n_kv_heads: int, head_dim: int, page_tokens: int, table=None,
                 scores=None, k_log2: int = 0, v_log2: int = 0):
        import torch
        page = lib().mk_kv4_page_bytes(n_kv_heads, head_dim, page_tokens)
        if page == 0:
            raise MkError(-9, "head_dim is 64 or 128, page_tokens a multiple of 32")
        if pool.dim() != 2 or lens.dim() != 1 or pool.shape[1] != page:
            raise ValueError(f"pool is [pages, {page}], lens [n_seq]")
        self.n_seq = lens.shape[0]
        if table is None:
            if self.n_seq == 0 or pool.shape[0] % self.n_seq:
                raise ValueError("without a table every sequence has the same number of pages")
            per = pool.shape[0] // self.n_seq
        else:
            if table.dim() != 2 or table.shape[0] != self.n_seq:
                raise ValueError("table is [n_seq, pages_per_seq]")
            per = table.shape[1]
        self.capacity = per * page_tokens
        self.n_kv_heads, self.head_dim, self.page_tokens = n_kv_heads, head_dim, page_tokens
        self.pool, self.lens, self.table, self.scores = pool, lens, table, scores
        self.device = d = pool.get_device()
        self.c = Kv4Struct(n_kv_heads, head_dim, page_tokens, pool.shape[0], self.n_seq, per, k_log2,
                           v_log2, _tensor(pool, torch.uint8, "pool"),
                           None if table is None else _tensor(table, torch.int32, "table", None, d),
                           _tensor(lens, torch.int32, "lens", None, d),
                           None if scores is None else _tensor(
                               scores, torch.float32, "scores", (self.n_seq, n_kv_heads, self.capacity), d))
        self.ref = C.addressof(self.c)


def _rows(t, heads, dim, what, device):
    """(pointer, elements between tokens, tokens) of token rows [tokens, heads,
    dim] whose heads lie together."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim or t.get_device() != device:
        raise ValueError(f"{what}: [tokens, {heads}, {dim}] on the cache's device expected, got {tuple(shape)}")
    n = shape[0]
    if t.is_contiguous():
        return t.data_ptr(), heads * dim, n
    st = t.stride()
    if st[2] != 1 or (heads > 1 and st[1] != dim):
        raise ValueError(f"{what}: a token's heads and dims are contiguous")
    return t.data_ptr(), st[0] if n > 1 else heads * dim, n


def kv4_append(cache: Kv4Cache, k, v, offsets, stream=None):
    """Packed new tokens k, v [tokens, n_kv_heads, head_dim] (token rows may be
    strided) into the cache; tokens offsets[s]..offsets[s+1] are the newest of
    sequence s, which cache.lens counts already (see mk_kv4_append)."""
    import torch
    d = cache.device
    kp, ks, n = _rows(k, cache.n_kv_heads, cache.head_dim, "k", d)
    vp, vs, m = _rows(v, cache.n_kv_heads, cache.head_dim, "v", d)
    code = _dtype(k)
    if n != m or _dtype(v) != code:
        raise ValueError("k and v have the same tokens and type")
    _on(d, stream, lib().mk_kv4_append, cache.ref, kp, vp, code, ks, vs,
        _tensor(offsets, torch.int32, "offsets", (cache.n_seq + 1,), d), n)


def kv4_read(cache: Kv4Cache, k_out, v_out, stream=None):
    """Values of slots [0, min(n, lens)) into k_out, v_out [n_seq, n,
    n_kv_heads, head_dim]; other rows are left (see mk_kv4_read)."""
    if k_out.dim() != 4:
        raise ValueError("k_out is [n_seq, n, n_kv_heads, head_dim]")
    n, d = k_out.shape[1], cache.device
    shape = (cache.n_seq, n, cache.n_kv_heads, cache.head_dim)
    _on(d, stream, lib().mk_kv4_read, cache.ref, _dtype(k_out), n, _tensor(k_out, None, "k_out", shape, d),
        _tensor(v_out, k_out.dtype, "v_out", shape, d))


def attention_kv4_workspace_bytes(cache: Kv4Cache, q_len: int, n_q_heads: int,
                                  accumulate: bool = False) -> int:
    return int(lib().mk_attention_kv4_workspace_bytes(cache.ref, q_len, n_q_heads, int(accumulate)))


def attention_kv4(cache: Kv4Cache, q, out, workspace, scale: Optional[float] = None,
                  accumulate: bool = False, stream=None):
    """Attention of the newest q_len tokens of every sequence, q and out
    [n_seq, q_len, n_q_heads, head_dim], over the cache; ``scale`` is
    1/sqrt(head_dim) unless given, ``accumulate`` adds the weights to
    cache.scores (see mk_attention_kv4)."""
    shape, d = q.shape, cache.device
    if len(shape) != 4 or shape[0] != cache.n_seq or shape[3] != cache.head_dim or q.get_device() != d:
        raise ValueError(f"q: [{cache.n_seq}, q_len, n_q_heads, {cache.head_dim}] on the cache's device "
                         f"expected, got {tuple(shape)}")
    n_seq, q_len, heads, dim = shape
    if q.is_contiguous():
        row = heads * dim
    else:
        st = q.stride()
        row = st[1] if q_len > 1 else (st[0] if n_seq > 1 else heads * dim)
        if st[3] != 1 or (heads > 1 and st[2] != dim) or (n_seq > 1 and st[0] != q_len * row):
            raise ValueError("q: a token's heads and dims are contiguous, tokens evenly spaced")
    _on(d, stream, lib().mk_attention_kv4, cache.ref, q.data_ptr(), _dtype(q), q_len, heads, row,
        dim ** -0.5 if scale is None else scale, accumulate, _tensor(workspace, None, "workspace", None, d),
        workspace.nbytes, _tensor(out, q.dtype, "out", shape, d))


def kv4_evict(src: Kv4Cache, dst: Kv4Cache, budget: int, keep_first: int, keep_last: int, kept,
              stream=None):
    """The rows of src that a budget leaves -- its ends and the highest scores
    -- into dst, their slots into kept int32 [n_seq, n_kv_heads, budget].
    Every slot that lens counts has a page, in src and, up to the budget, in
    dst (see mk_kv4_evict)."""
    import torch
    d = src.device
    if dst.device != d:
        raise ValueError(f"caches on devices {d} and {dst.device}")
    _on(d, stream, lib().mk_kv4_evict, src.ref, dst.ref, budget, keep_first, keep_last,
        _tensor(kept, torch.int32, "kept", (src.n_seq, src.n_kv_heads, budget), d))


def kv4_reorder(cache: Kv4Cache, parents, first: int, n_keys: int, stream=None):
    """Reorders the sequences of each search in place: parents int32
    [n_seq / beams, beams] (see mk_kv4_reorder)."""
    import torch
    if parents.dim() != 2 or parents.numel() != cache.n_seq:
        raise ValueError("parents is [searches, beams], one entry per sequence")
    d = cache.device
    _on(d, stream, lib().mk_kv4_reorder, cache.ref, _tensor(parents, torch.int32, "parents", None, d),
        parents.shape[1], first, n_keys)


def beam_select_workspace_bytes(n_batch: int, beams: int, vocab: int) -> int:
    return int(lib().mk_beam_select_workspace_bytes(n_batch, beams, vocab))


def beam_select(logits, cum, tokens, parents, scores, workspace, finished=None, finished_out=None,
                eos: int = -1, stream=None):
    """The next beams of every search: logits [n_batch * beams, vocab] (rows may
    be strided), cum fp32 [n_batch, beams] -> tokens, parents int32, scores
    fp32 and finished_out (bool or uint8), all [n_batch, beams] (see
    mk_beam_select)."""
    import torch
    shape, d = cum.shape, logits.get_device()
    if len(shape) != 2 or logits.dim() != 2 or logits.shape[0] != shape[0] * shape[1]:
        raise ValueError("cum is [n_batch, beams], logits [n_batch * beams, vocab]")
    rows, vocab = logits.shape
    st = logits.stride()
    if d < 0 or (vocab > 1 and st[1] != 1):
        raise ValueError("logits: CUDA, contiguous rows")
    flags = (torch.bool, torch.uint8)
    if (finished is not None and finished.dtype not in flags) or \
            (finished_out is not None and finished_out.dtype not in flags):
        raise TypeError("finished flags are bool or uint8")
    _on(d, stream, lib().mk_beam_select, logits.data_ptr(), _dtype(logits), st[0] if rows > 1 else vocab,
        _tensor(cum, torch.float32, "cum", None, d),
        None if finished is None else _tensor(finished, None, "finished", shape, d), shape[0], shape[1],
        vocab, eos, _tensor(tokens, torch.int32, "tokens", shape, d),
        _tensor(parents, torch.int32, "parents", shape, d), _tensor(scores, torch.float32, "scores", shape, d),
        None if finished_out is None else _tensor(finished_out, None, "finished_out", shape, d),
        _tensor(workspace, None, "workspace", None, d), workspace.nbytes)


def beam_reorder(state, parents, first: int, count: int, stream=None):
    """Reorders states [n_batch * beams, segments, positions, ...] (contiguous,
    any type) in place by parents int32 [n_batch, beams]; positions [first,
    first + count) of every segment move, the others stay (see
    mk_beam_reorder)."""
    import torch
    base, d = _tensor(state, None, "state"), state.get_device()
    if state.dim() < 3 or parents.dim() != 2 or parents.numel() != state.shape[0]:
        raise ValueError("state is [n_batch * beams, segments, positions, ...], parents [n_batch, beams]")
    segments, positions = state.shape[1], state.shape[2]
    if first < 0 or count < 0 or first + count > positions:
        raise ValueError("positions [first, first + count) of the state")
    if count == 0 or state.numel() == 0:
        return
    row = state.nbytes // (state.shape[0] * segments * positions)   # not a stride: of one position it may be anything
    _on(d, stream, lib().mk_beam_reorder, base + first * row, _tensor(parents, torch.int32, "parents", None, d),
        parents.shape[0], parents.shape[1], segments * positions * row, segments, positions * row, count * row)
