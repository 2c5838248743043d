"""Device state of a generation over the 4-bit cache: its planes, row counts, workspaces and the calls
that use them (``spatten_prompt_attention``, ``spatten_kv4_append`` / ``_attention`` / ``_evict`` /
``_read``).  Argument marshalling only -- every step runs in the library's kernels.

    st = KV4State(B, H, H_kv, d_h, cap)
    o = st.prompt(q, k, v, cu)             # causal attention of packed prompts; fills the cache
    st.evict(keep, recent)                 # keep the rows with the most accumulated weight
    o = st.step(q, k, v)                   # one token per sequence: append, attend
    o = st.resume(q, k, v, cu, cu_kv, rows)   # prompts that go on over the cached rows

Calls run on the state's GPU, on torch's current stream there.  The counts live on the device, so ``step`` and ``evict`` can be
captured in a CUDA graph and replayed.
"""
import ctypes as C

import torch

from . import spatten as S


class KV4State:
    """A cache of ``cap`` rows per (sequence, key/value head) for ``B`` sequences of ``H`` query heads.

    Tensors a caller may look at: ``k_codes``, ``k_scale``, ``v_codes``, ``v_scale`` (the planes),
    ``weight`` (accumulated attention weight), ``pos`` (token positions), ``len`` (rows held), ``seen``
    (next position), ``status`` (first device-side error, 0 = none)."""

    def __init__(self, B, H, H_kv, d_h, cap, device="cuda"):
        if not 1 <= H <= 1024 or H_kv < 1 or H % H_kv or d_h not in (64, 128):
            raise ValueError("H is a multiple of H_kv, up to 1024, and d_h 64 or 128")
        self.B, self.H, self.H_kv, self.d_h, self.cap = B, H, H_kv, d_h, cap
        z = lambda *shape, dt: torch.zeros(shape, dtype=dt, device=device)
        self.k_codes, self.v_codes = (z(B, H_kv, cap, d_h // 2, dt=torch.uint8) for _ in range(2))
        self.k_scale, self.v_scale = (z(B, H_kv, cap, d_h // 32, dt=torch.bfloat16) for _ in range(2))
        self.weight, self.pos = z(B, H_kv, cap, dt=torch.float32), z(B, H_kv, cap, dt=torch.int32)
        self.len, self.seen = z(B, dt=torch.int32), z(B, dt=torch.int32)
        self.status = z(1, dt=torch.int32)
        self.cache = S.make_kv4_cache(self.k_codes, self.k_scale, self.v_codes, self.v_scale, self.weight, self.pos)
        self._ws = {}

    def _workspace(self, key, nbytes):
        """A workspace of the state's own for one kind of call: calls of one state run in order.  One that
        becomes too small stays alive, since a captured graph may hold its address (or another stream still use
        it); the next one is at least twice as large, so that all of them stay below four times the largest need."""
        held = self._ws.setdefault(key, [])
        if not held or held[-1].numel() < nbytes:
            size = max(nbytes, 256, 2 * held[-1].numel() if held else 0)
            held.append(torch.empty(size, dtype=torch.uint8, device=self.k_codes.device))
        return held[-1]

    def append(self, k, v, cu=None):
        """Quantize rows k, v [rows, H_kv, d_h] behind each sequence's rows (cu None: one row each)."""
        if k.shape != v.shape or k.stride() != v.stride() or tuple(k.shape[1:]) != (self.H_kv, self.d_h) or (
                k.stride(2) != 1 or (self.H_kv > 1 and k.stride(1) != self.d_h)):
            raise ValueError("k and v are [rows, H_kv, d_h] alike, with the heads of a row contiguous")
        if k.dtype != v.dtype:
            raise TypeError("k and v have one dtype")
        if cu is not None and S._i32_vector(cu, "cu") != self.B + 1:
            raise ValueError("cu has one entry more than there are sequences")
        if cu is None and k.shape[0] != self.B:
            raise ValueError("without cu there is one row per sequence")
        S.kv4_append(self.cache, k, v, S._row_stride(k), k.shape[0], self.len, self.len, self.seen, self.seen, cu=cu,
                     dev_status=self.status)

    def prompt(self, q, k, v, cu, o=None):
        """Causal attention of packed prompts (rows cu[b] .. cu[b+1]-1 are sequence b's) into an empty
        cache: returns the outputs, appends the rows and adds their attention weights.  A sequence of
        which the cache held rows is reported (``status``) and adds no weights."""
        o, *call = self._prepare(q, k, v, cu, None, o)
        self.append(k, v, cu)
        S.prompt_attention(*call)
        return o

    def resume(self, q, k, v, cu, cu_kv, rows, o=None):
        """Packed prompts that go on over the cached rows.  cu_kv [B + 1] are the offsets of each
        sequence's cached and new rows together, ``rows`` their number in all.  Every row, the new ones
        too, takes part as the value its codes stand for.  A sequence whose rows are not as many as
        cu_kv says is reported (``status``) and adds no weights."""
        if cu_kv is None:
            raise ValueError("cu_kv has the offsets of each sequence's cached and new rows together")
        kk, vv = (torch.zeros((rows, self.H_kv, self.d_h), dtype=q.dtype, device=q.device) for _ in range(2))
        o, *call = self._prepare(q, kk, vv, cu, cu_kv, o)
        self.append(k, v, cu)
        S.kv4_read(self.cache, cu_kv, rows, kk, vv, self.H_kv * self.d_h, dev_status=self.status)
        S.prompt_attention(*call)
        return o

    def _prepare(self, q, k, v, cu, cu_kv, o):
        """A prompt's outputs, arguments and workspace.  What the call would refuse is refused here, before its
        rows are appended."""
        o = torch.empty_like(q) if o is None else o
        a = S.make_prompt_args(q, k, v, o, cu, cu_kv, weight=self.weight, dev_status=self.status,
                               weight_len=self.len)
        # made without its workspace, which one with weights needs and which is looked at last, it launches nothing
        status = S.lib.spatten_prompt_attention(C.byref(a), None, 0, None)
        if status != S.E_WORKSPACE:
            S.check(status, "spatten_prompt_attention")
        nb = S.prompt_workspace_size(a)
        return o, a, self._workspace("prompt", nb), nb

    def attend(self, q, o=None, n_max=None, update_weight=True):
        """Attention of one query row per sequence, q [B, H, d_h], over the cached rows."""
        o, *call = self._prepare_row(q, o, n_max, update_weight)
        S.kv4_attention(*call)
        return o

    def step(self, q, k, v, o=None, n_max=None):
        """One token per sequence: append its key and value rows [B, H_kv, d_h], then attend."""
        o, *call = self._prepare_row(q, o, n_max, True)
        self.append(k, v)
        S.kv4_attention(*call)
        return o

    def _prepare_row(self, q, o, n_max, update_weight):
        o = torch.empty_like(q) if o is None else o
        a = S.make_kv4_attn_args(self.cache, q, o, self.len, self.cap if n_max is None else n_max, update_weight,
                                 dev_status=self.status)
        nb = S.kv4_attention_workspace_size(a)
        if nb == 0:   # the call says what is wrong with it
            S.check(S.lib.spatten_kv4_attention(C.byref(a), None, 0, None), "spatten_kv4_attention")
        return o, a, self._workspace("attend", nb), nb

    def evict(self, keep, recent=0, n_max=None):
        """Keep each head's ``keep`` rows with the most accumulated weight (and the last ``recent``)."""
        n_max = self.cap if n_max is None else n_max
        nb = S.kv4_evict_workspace_size(self.cache, n_max, keep)
        S.kv4_evict(self.cache, self.cache, self.len, self.len, self.seen, n_max, keep, recent,
                    self._workspace("evict", nb), nb, self.status)
