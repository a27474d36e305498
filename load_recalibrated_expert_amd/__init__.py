"""Memory-aware MoE expert backward (LRMoE) on MI355X: Python binding of liblrmoe.

The five steps of the LRMoE paper's backward-time calibration (Algorithm 1,
section 3.3) are calls into ``liblrmoe.so`` (hand-written HIP for gfx950):

    score -> select -> compact_weighted -> grouped_gemm_bwd_gathered -> scatter

(or, packing the weighted gradient rows instead, compact -> grouped_gemm_bwd).

The functions here have the C entry points' names and only marshal arguments:
torch tensors supply device memory and the current HIP stream. ``backward`` chains
the five calls. ``Checkpoint`` holds saved activations in 8 bits: expert_forward_checkpoint
(or checkpoint) makes one, and backward takes it in the place of H and Phi, and of X. Around the
experts, ``Router`` with route, balance_loss, alpha_grad and route_bwd makes the pair lists and trains
the router, bias_update balances it, and ``AdamW`` applies the gradients.
Nothing falls back to another implementation; if the library is not built, the first call
raises ImportError.
"""
from __future__ import annotations

import bisect
import ctypes

import numpy as np
import torch

from . import _lib
from ._lib import (BF16, COMPACT_PHYSICAL, COMPACT_ZERO_MASKED, F32, SCATTER_SLOT, SCATTER_TOKEN,
                   SCATTER_TOKEN_BESIDE,
                   InfeasibleQuotaError, LrmoeError)

__all__ = ["Problem", "score", "select", "select_noalloc", "compact", "compact_weighted", "grouped_gemm_bwd",
           "grouped_gemm_bwd_gathered", "expert_forward", "scatter", "backward", "backward_bytes", "plan_quotas",
           "Checkpoint", "checkpoint", "restore", "expert_forward_checkpoint", "score_checkpoint", "compact_checkpoint",
           "grouped_gemm_bwd_checkpoint", "Router", "route", "bias_update", "balance_loss", "route_bwd", "alpha_grad", "AdamW", "library", "BF16", "F32", "COMPACT_PHYSICAL", "COMPACT_ZERO_MASKED", "SCATTER_TOKEN",
           "SCATTER_SLOT", "SCATTER_TOKEN_BESIDE", "LrmoeError", "InfeasibleQuotaError"]


def library() -> ctypes.CDLL:
    return _lib.load()


def _ptr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to liblrmoe must be contiguous")
    return t.data_ptr()


def _stream(stream=None):
    here = torch._C._cuda_getDevice()
    if stream is not None:
        if stream.device_index != here:
            raise ValueError(f"stream: of cuda:{stream.device_index}, which is not the current device")
        return stream.cuda_stream
    # the handle alone: a torch.cuda.Stream object costs 3 us of host time per call
    return torch._C._cuda_getCurrentRawStream(here)


def _event(ev, stream=None):
    """Raw handle of a torch.cuda.Event (None -> NULL). torch creates the HIP event on its
    first record, so an event never recorded is recorded once here, on `stream`."""
    if ev is None:
        return None
    if not ev.cuda_event:
        ev.record(stream if stream is not None else torch.cuda.current_stream())
    return ev.cuda_event


class Problem:
    """Shapes, pair segments and quotas of one layer invocation (host + device copies).

    seg_off: int64 [E+1] pair offsets per expert (pairs stored expert-major);
    quota: int32 [E] retention quotas, fixed before the call."""

    def __init__(self, *, E, T, K, D, F, swiglu, dtype, seg_off, quota, device="cuda"):
        lib = library()
        self.E, self.T, self.K, self.D, self.F = int(E), int(T), int(K), int(D), int(F)
        self.swiglu, self.dtype = bool(swiglu), int(dtype)
        self.c, self._keep = _lib.make_problem_struct(self.E, self.T, self.K, self.D, self.F, self.swiglu,
                                                      self.dtype, seg_off, quota)
        k_tot = ctypes.c_int64(0)
        cseg = np.zeros(self.E + 1, dtype=np.int64)
        _lib.check(lib.lrmoe_validate(ctypes.byref(self.c), ctypes.byref(k_tot),
                                      cseg.ctypes.data_as(ctypes.POINTER(ctypes.c_int64))), "lrmoe_validate")
        self.N = int(self._keep[0][-1])
        self.K_tot = int(k_tot.value)
        self.seg_off = self._keep[0]
        self.quota = self._keep[1]
        self.cseg_off = cseg
        self.device = torch.device(device)
        self.seg_off_d = torch.from_numpy(self.seg_off).to(self.device)
        self.quota_d = torch.from_numpy(self.quota).to(self.device)
        self.cseg_off_d = torch.from_numpy(self.cseg_off).to(self.device)
        self._ws = None
        self._ws_size = {}

    @property
    def torch_dtype(self):
        return torch.bfloat16 if self.dtype == BF16 else torch.float32

    def workspace_size(self, mode=COMPACT_PHYSICAL) -> int:
        """lrmoe_workspace_size, asked once per mode (the quotas are fixed for the problem)."""
        if mode not in self._ws_size:
            n = ctypes.c_size_t(0)
            _lib.check(library().lrmoe_workspace_size(ctypes.byref(self.c), mode, ctypes.byref(n)),
                       "lrmoe_workspace_size")
            self._ws_size[mode] = int(n.value)
        return self._ws_size[mode]

    def workspace(self, mode=COMPACT_PHYSICAL) -> torch.Tensor:
        """The problem's scratch buffer, large enough for every call in ``mode`` (it grows
        once when a zero-masked call needs more than the physical ones)."""
        n = self.workspace_size(mode)
        if self._ws is None or self._ws.numel() < n:
            self._ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        return self._ws

    def rows(self, mode=COMPACT_PHYSICAL) -> int:
        return self.K_tot if mode == COMPACT_PHYSICAL else self.N

    def row_off_d(self, mode=COMPACT_PHYSICAL):
        return self.cseg_off_d if mode == COMPACT_PHYSICAL else self.seg_off_d


def _restored_bytes(T, D, dtype, restored_x):
    """The rows of X that ``backward`` restores from a Checkpoint, whatever the quotas."""
    return int(T) * int(D) * (2 if dtype == BF16 else 4) if restored_x else 0


def backward_bytes(p: Problem, packed=False, restored_x=False) -> int:
    """Device bytes one physical-compaction backward holds at p's quotas besides its
    inputs: its buffers and its workspace (host-only; the list is in the header,
    lrmoe_backward_bytes). ``restored_x``: X is a Checkpoint, whose rows the backward holds too."""
    n = ctypes.c_size_t(0)
    _lib.check(library().lrmoe_backward_bytes(ctypes.byref(p.c), int(bool(packed)), ctypes.byref(n)),
               "lrmoe_backward_bytes")
    return int(n.value) + _restored_bytes(p.T, p.D, p.dtype, restored_x)


def plan_quotas(E, T, K, D, F, swiglu, dtype, seg_off, rhos, hbm_avail, packed=False, restored_x=False):
    """Quota admission on one GPU (host-only): the largest candidate ratio in ``rhos``
    (exact decimals such as "0.6", or Fractions) whose backward (buffers and workspace)
    fits ``hbm_avail`` bytes. Returns (index into rhos, quotas [E] int32, bytes); raises InfeasibleQuotaError
    when none fits (Algorithm 1's "return Infeasible"). ``restored_x``: as in backward_bytes."""
    from fractions import Fraction
    restored = _restored_bytes(T, D, dtype, restored_x)
    if restored:  # no estimate is 0 bytes
        hbm_avail = max(int(hbm_avail) - restored, 0)
    fr = [Fraction(r) for r in rhos]
    num = np.array([f.numerator for f in fr], dtype=np.int32)
    den = np.array([f.denominator for f in fr], dtype=np.int32)
    c, keep = _lib.make_problem_struct(E, T, K, D, F, swiglu, dtype, seg_off, np.zeros(E, dtype=np.int32))
    chosen, nb = ctypes.c_int32(-1), ctypes.c_size_t(0)
    q = np.zeros(E, dtype=np.int32)
    I32 = ctypes.POINTER(ctypes.c_int32)
    _lib.check(library().lrmoe_plan_quotas(ctypes.byref(c), num.ctypes.data_as(I32), den.ctypes.data_as(I32),
                                           len(fr), int(bool(packed)), int(hbm_avail), ctypes.byref(chosen),
                                           q.ctypes.data_as(I32), ctypes.byref(nb)), "lrmoe_plan_quotas")
    return int(chosen.value), q, int(nb.value) + restored


CRITERIA = {"lrm": 0, "grad_sqnorm": 1, "grad_abs": 2}


def score(p: Problem, G, Phi, alpha, tok, R=None, criterion="lrm", stream=None):
    """Step 1. ``criterion``: "lrm" (the LRM score), or the gradient-only criteria of the
    ablation, "grad_sqnorm" / "grad_abs" (Phi and alpha may then be None)."""
    R = R if R is not None else torch.empty(p.N, dtype=torch.float32, device=p.device)
    ws = p.workspace()
    if criterion == "lrm":
        _lib.check(library().lrmoe_score(ctypes.byref(p.c), _ptr(G), _ptr(Phi), _ptr(alpha), _ptr(tok), _ptr(R),
                                         _ptr(ws), ws.numel(), _stream(stream)), "lrmoe_score")
    else:
        if criterion not in CRITERIA:
            raise ValueError(f"unknown criterion {criterion!r}; expected one of {sorted(CRITERIA)}")
        _lib.check(library().lrmoe_score_criterion(ctypes.byref(p.c), CRITERIA[criterion], _ptr(G), _ptr(Phi),
                                                   _ptr(alpha), _ptr(tok), _ptr(R), _ptr(ws), ws.numel(),
                                                   _stream(stream)), "lrmoe_score_criterion")
    return R


def select(p: Problem, R, sel=None, keep=None, want_keep=True, tok=None, slot=None, maps=None, stream=None):
    """Step 2. Returns (sel, keep). With the pairs' ``tok`` and ``slot`` it also writes the
    (token, slot) -> packed row map and the packed rows' tokens and slots, and returns
    (sel, keep, maps) with maps = {"pmap", "ctok", "cslot"} (``maps`` reuses buffers)."""
    sel = sel if sel is not None else torch.empty(max(p.K_tot, 1), dtype=torch.int32, device=p.device)
    if keep is None and want_keep:
        keep = torch.empty(max(p.N, 1), dtype=torch.uint8, device=p.device)
    m = None
    if tok is not None:
        m = dict(maps or {})
        m.setdefault("pmap", torch.empty(max(p.T * p.K, 1), dtype=torch.int32, device=p.device))
        m.setdefault("ctok", torch.empty(max(p.K_tot, 1), dtype=torch.int32, device=p.device))
        m.setdefault("cslot", torch.empty(max(p.K_tot, 1), dtype=torch.int32, device=p.device))
    ws = p.workspace()
    _lib.check(library().lrmoe_select(ctypes.byref(p.c), _ptr(R), _ptr(p.seg_off_d), _ptr(p.quota_d),
                                      _ptr(p.cseg_off_d), _ptr(sel), _ptr(keep), _ptr(tok), _ptr(slot),
                                      _ptr(m["pmap"]) if m else None, _ptr(m["ctok"]) if m else None,
                                      _ptr(m["cslot"]) if m else None, _ptr(ws), ws.numel(), _stream(stream)),
               "lrmoe_select")
    out = (sel[:p.K_tot], (keep[:p.N] if keep is not None else None))
    if m is None:
        return out
    return out + ({"pmap": m["pmap"][:p.T * p.K], "ctok": m["ctok"][:p.K_tot], "cslot": m["cslot"][:p.K_tot]},)


def select_noalloc(p: Problem, R, sel, keep=None, tok=None, slot=None, maps=None, stream=None):
    """lrmoe_select_noalloc: step 2 with the library's fixed per-GPU scratch instead of a
    workspace, for callers that cannot allocate. The caller passes every output (``sel``
    [K_tot], optional ``keep`` [N]; with ``tok``/``slot`` also ``maps`` = {"pmap", "ctok",
    "cslot"}); nothing is allocated here."""
    m = maps if tok is not None else None
    _lib.check(library().lrmoe_select_noalloc(ctypes.byref(p.c), _ptr(R), _ptr(p.seg_off_d), _ptr(p.quota_d),
                                              _ptr(p.cseg_off_d), _ptr(sel), _ptr(keep), _ptr(tok), _ptr(slot),
                                              _ptr(m["pmap"]) if m else None, _ptr(m["ctok"]) if m else None,
                                              _ptr(m["cslot"]) if m else None, _stream(stream)),
               "lrmoe_select_noalloc")
    return sel, keep, m


def compact(p: Problem, G, Phi, alpha, tok, slot, sel=None, keep=None, X=None, H=None,
            mode=COMPACT_PHYSICAL, out=None, pack_phi=True, maps=None, stream=None):
    """Always writes Dlt; ctok/cslot too unless ``maps`` (the map, ctok and cslot that
    select wrote for this sel) is given, in which case they are returned as given and the
    gather runs through that map. The saved rows are packed only on request: PhiC when
    ``pack_phi`` (physical mode), XC when X is given, HC when H is given (physical mode).
    The grouped GEMM can read each of them in place instead, through its row maps (sel for
    Phi and H, ctok or tok for X)."""
    rows = p.rows(mode)
    dt = p.torch_dtype
    o = dict(out or {})
    dev = p.device
    o.setdefault("Dlt", torch.empty(max(rows, 1), p.D, dtype=dt, device=dev))
    if mode == COMPACT_PHYSICAL:
        if pack_phi:
            o.setdefault("PhiC", torch.empty(max(rows, 1), p.F, dtype=dt, device=dev))
        if p.swiglu and H is not None:
            o.setdefault("HC", torch.empty(max(rows, 1), 2 * p.F, dtype=dt, device=dev))
    if p.swiglu and X is not None:
        o.setdefault("XC", torch.empty(max(rows, 1), p.D, dtype=dt, device=dev))
    pmap = None
    if maps is not None:
        o["ctok"], o["cslot"], pmap = maps["ctok"], maps["cslot"], maps["pmap"]
    else:
        o.setdefault("ctok", torch.empty(max(rows, 1), dtype=torch.int32, device=dev))
        o.setdefault("cslot", torch.empty(max(rows, 1), dtype=torch.int32, device=dev))
    ws = p.workspace()
    _lib.check(library().lrmoe_compact(
        ctypes.byref(p.c), mode, _ptr(sel), _ptr(keep), _ptr(G), _ptr(Phi), _ptr(X), _ptr(H), _ptr(alpha),
        _ptr(tok), _ptr(slot), _ptr(o["Dlt"]), _ptr(o.get("PhiC")), _ptr(o.get("XC")), _ptr(o.get("HC")),
        _ptr(o["ctok"]), _ptr(o["cslot"]), _ptr(pmap), _ptr(ws), ws.numel(), _stream(stream)), "lrmoe_compact")
    return {k: v[:rows] for k, v in o.items()}


def grouped_gemm_bwd(p: Problem, Dlt, PhiC, W2, XC=None, HC=None, W1=None, mode=COMPACT_PHYSICAL,
                     out=None, accumulate=False, hc_rows=None, phi_rows=None, x_rows=None, din_ready=None,
                     stream=None):
    """``PhiC``, ``XC`` and ``HC`` are packed rows, or the saved matrices themselves (Phi,
    X, H) with a row map giving, for each packed row, the row to read: ``phi_rows`` and
    ``hc_rows`` index pair rows (e.g. ``sel``), ``x_rows`` token rows (``ctok``, or ``tok``
    in zero-masked mode). ``din_ready`` (a torch.cuda.Event) is recorded on the stream as
    soon as dIn is complete, before the weight-gradient launches."""
    rows = p.rows(mode)
    dt = p.torch_dtype
    dev = p.device
    o = dict(out or {})
    o.setdefault("dW2", torch.empty(p.E, p.F, p.D, dtype=torch.float32, device=dev))
    if p.swiglu:
        o.setdefault("dW1", torch.empty(p.E, p.D, 2 * p.F, dtype=torch.float32, device=dev))
        o.setdefault("dH", torch.empty(max(rows, 1), 2 * p.F, dtype=dt, device=dev))
        o.setdefault("dIn", torch.empty(max(rows, 1), p.D, dtype=dt, device=dev))
    else:
        o.setdefault("dIn", torch.empty(max(rows, 1), p.F, dtype=dt, device=dev))
    ws = p.workspace(mode)
    _lib.check(library().lrmoe_grouped_gemm_bwd(
        ctypes.byref(p.c), mode, _ptr(p.row_off_d(mode)), _ptr(Dlt), _ptr(PhiC), _ptr(XC), _ptr(HC), _ptr(hc_rows),
        _ptr(phi_rows), _ptr(x_rows), _ptr(W2),
        _ptr(W1), _ptr(o["dW2"]), _ptr(o.get("dW1")), _ptr(o.get("dH")), _ptr(o["dIn"]), int(bool(accumulate)),
        _ptr(ws), ws.numel(), _stream(stream), _event(din_ready, stream)), "lrmoe_grouped_gemm_bwd")
    res = dict(o)
    res["dIn"] = o["dIn"][:rows]
    if "dH" in o:
        res["dH"] = o["dH"][:rows]
    return res


def compact_weighted(p: Problem, sel, Phi, alpha, out=None, stream=None):
    """Step 3 for the path that reads gradient rows by token: PhiW[c] = alpha[sel[c]] *
    Phi[sel[c]] over the K_tot packed rows (lrmoe_compact_weighted)."""
    PhiW = out if out is not None else torch.empty(max(p.K_tot, 1), p.F, dtype=p.torch_dtype, device=p.device)
    _lib.check(library().lrmoe_compact_weighted(ctypes.byref(p.c), _ptr(sel), _ptr(Phi), _ptr(alpha), _ptr(PhiW),
                                                _stream(stream)), "lrmoe_compact_weighted")
    return PhiW[:p.K_tot]


def _gemm_outputs(p, rows, out):
    """The outputs of the gathered grouped GEMM, those that `out` does not give allocated."""
    dt, dev = p.torch_dtype, p.device
    o = dict(out or {})
    o.setdefault("dW2", torch.empty(p.E, p.F, p.D, dtype=torch.float32, device=dev))
    if p.swiglu:
        o.setdefault("dW1", torch.empty(p.E, p.D, 2 * p.F, dtype=torch.float32, device=dev))
        o.setdefault("dH", torch.empty(max(rows, 1), 2 * p.F, dtype=dt, device=dev))
        o.setdefault("dIn", torch.empty(max(rows, 1), p.D, dtype=dt, device=dev))
    else:
        o.setdefault("dIn", torch.empty(max(rows, 1), p.F, dtype=dt, device=dev))
    return o


def _gemm_results(p, rows, o):
    res = dict(o)
    res["dIn"] = o["dIn"][:rows]
    if "dH" in o:
        res["dH"] = o["dH"][:rows]
    return res


def grouped_gemm_bwd_gathered(p: Problem, G, alpha, sel, ctok, PhiW, W2, X=None, H=None, W1=None, out=None,
                              accumulate=False, din_ready=None, stream=None):
    """Step 4 without a packed Dlt (lrmoe_grouped_gemm_bwd_gathered): gradient rows G[ctok]
    and X[ctok] read by token, H[sel] and alpha[sel] by pair, PhiW from compact_weighted.
    Same outputs as grouped_gemm_bwd in physical mode."""
    o = _gemm_outputs(p, p.K_tot, out)
    ws = p.workspace(COMPACT_PHYSICAL)
    _lib.check(library().lrmoe_grouped_gemm_bwd_gathered(
        ctypes.byref(p.c), _ptr(p.cseg_off_d), _ptr(G), _ptr(alpha), _ptr(sel), _ptr(ctok), _ptr(PhiW), _ptr(X),
        _ptr(H), _ptr(W2), _ptr(W1), _ptr(o["dW2"]), _ptr(o.get("dW1")), _ptr(o.get("dH")), _ptr(o["dIn"]),
        int(bool(accumulate)), _ptr(ws), ws.numel(), _stream(stream), _event(din_ready, stream)),
        "lrmoe_grouped_gemm_bwd_gathered")
    return _gemm_results(p, p.K_tot, o)


def expert_forward(p: Problem, X, tok, alpha, W1, W2, out=None, stream=None):
    """The forward that saves the backward's context: H = X[tok] W1 ([gate | up]),
    Phi = silu(gate) * up, Y = alpha * Phi W2 (rows of the N pairs, expert-major).
    The layer output is ``scatter(p, Y, tok, slot, n_rows=p.N)``."""
    dt = torch.bfloat16
    o = out or {}
    H = o.get("H") if o.get("H") is not None else torch.empty(max(p.N, 1), 2 * p.F, dtype=dt, device=p.device)
    Phi = o.get("Phi") if o.get("Phi") is not None else torch.empty(max(p.N, 1), p.F, dtype=dt, device=p.device)
    Y = o.get("Y") if o.get("Y") is not None else torch.empty(max(p.N, 1), p.D, dtype=dt, device=p.device)
    _lib.check(library().lrmoe_expert_forward(ctypes.byref(p.c), _ptr(p.seg_off_d), _ptr(X), _ptr(tok), _ptr(alpha),
                                              _ptr(W1), _ptr(W2), _ptr(H), _ptr(Phi), _ptr(Y), _stream(stream)),
               "lrmoe_expert_forward")
    return {"H": H[:p.N], "Phi": Phi[:p.N], "Y": Y[:p.N]}


def scatter(p: Problem, rows_t, ctok, cslot, n_rows=None, mode=SCATTER_TOKEN, out=None, ws=None, pmap=None,
            stream=None):
    """``pmap``: the (token, slot) map select wrote for these packed rows (then no workspace
    is used). Without it the map is built in ``ws``, which defaults to the problem's
    workspace; a scatter running concurrently with another call of the same problem (on
    another stream) then needs its own."""
    n_rows = rows_t.shape[0] if n_rows is None else n_rows
    width = rows_t.shape[1]
    rdt = BF16 if rows_t.dtype == torch.bfloat16 else F32
    if out is None:
        nout = p.T if mode in (SCATTER_TOKEN, SCATTER_TOKEN_BESIDE) else p.T * p.K
        out = torch.empty(max(nout, 1), width, dtype=torch.float32, device=p.device)
    if pmap is None:
        ws = p.workspace() if ws is None else ws
    _lib.check(library().lrmoe_scatter(ctypes.byref(p.c), mode, n_rows, width, rdt, _ptr(rows_t), _ptr(ctok),
                                       _ptr(cslot), _ptr(pmap), _ptr(out), _ptr(ws), 0 if ws is None else ws.numel(),
                                       _stream(stream)), "lrmoe_scatter")
    return out


def _saved_in_8_bits(p, Phi, H):
    """The Checkpoint that phi comes from, or None."""
    if isinstance(H, Checkpoint):
        if not p.swiglu or Phi is not None:
            raise ValueError("a checkpoint of [gate | up] is for SwiGLU problems, without Phi")
        return H
    if isinstance(Phi, Checkpoint):
        if p.swiglu:
            raise ValueError("a SwiGLU problem takes a checkpoint of [gate | up], not of Phi")
        return Phi
    if Phi is None and p.N:  # without pairs there are no rows to give
        raise ValueError("Phi is missing")
    return None


def backward(p: Problem, *, G, Phi=None, alpha, tok, slot, W2, X=None, H=None, W1=None, mode=COMPACT_PHYSICAL,
             scatter_mode=SCATTER_TOKEN, bufs=None, overlap_scatter=False, packed_dlt=False, stream=None):
    """The whole path: score -> select -> compact -> grouped GEMMs -> scatter.

    Physical compaction packs only the weighted saved rows PhiW = alpha Phi[sel] and the
    grouped GEMMs read the gradient rows G[ctok], the FC1 inputs X[ctok] and the saved
    [gate | up] rows H[sel] in place (compact_weighted, grouped_gemm_bwd_gathered). With
    ``packed_dlt`` (and always in zero-masked mode) compaction packs the weighted gradient
    rows Dlt instead and grouped_gemm_bwd reads them.

    Saved activations in 8 bits: ``H`` may be a Checkpoint of the [gate | up] rows (``Phi`` is then left out), or
    ``Phi`` one of the Phi rows of an FC2-only problem, and ``X`` one of the FC1 inputs, which are restored for the
    call (``backward_bytes`` counts them with ``restored_x``). Physical compaction without ``packed_dlt`` only.

    ``bufs`` (a dict, optional) carries preallocated outputs between calls; it is
    filled on first use. With ``overlap_scatter`` the scatter runs on a second stream as
    soon as the input gradients are complete, while the weight gradients are computed
    (with a workspace of its own when it builds its map); the calling stream waits for it
    before returning. A token-order scatter then uses SCATTER_TOKEN_BESIDE, whose blocks
    share the compute units the weight-gradient launch occupies (same results, bit for
    bit). Returns a dict of every intermediate and output."""
    b = bufs if bufs is not None else {}
    main = stream if stream is not None else torch.cuda.current_stream()
    phys = mode == COMPACT_PHYSICAL
    saved = _saved_in_8_bits(p, Phi, H)
    if isinstance(X, Checkpoint) or saved is not None:
        if not phys or packed_dlt:
            raise ValueError("checkpoints need physical compaction without packed_dlt")
        if isinstance(X, Checkpoint):
            if not p.swiglu:
                raise ValueError("FC2-only problems take no X")
            X._ptrs("X", p.T, 1, p.D, torch._C._cuda_getDevice())
    if saved is None:
        b["R"] = score(p, G, Phi, alpha, tok, R=b.get("R"), stream=stream)
    else:
        b["R"] = score_checkpoint(p, G, saved, alpha, tok, R=b.get("R"), stream=stream)
    maps = None
    if phys:  # the selection also writes the (token, slot) map that compaction and the scatter use
        sel, keep, maps = select(p, b["R"], sel=b.get("sel_full"), keep=b.get("keep_full"), tok=tok, slot=slot,
                                 maps=b.get("maps"), stream=stream)
        b.setdefault("maps", maps)
    else:
        sel, keep = select(p, b["R"], sel=b.get("sel_full"), keep=b.get("keep_full"), stream=stream)
    b.setdefault("sel_full", sel)
    b.setdefault("keep_full", keep)
    gathered = phys and not packed_dlt
    if gathered:  # the weighted saved rows only; G, X and H are read in place
        if saved is None:
            PhiW = compact_weighted(p, sel, Phi, alpha, out=b.get("PhiW"), stream=stream)
        else:
            PhiW = compact_checkpoint(p, sel, saved, alpha, out=b.get("PhiW"), stream=stream)
        if isinstance(X, Checkpoint):
            rows = Checkpoint._of(X.q[:p.T], X.scale[:p.T], 1, p.D)
            X = b["X"] = restore(rows, dtype=p.torch_dtype, out=b.get("X"), stream=stream)
        b.setdefault("PhiW", PhiW)
        c = {"PhiW": PhiW, "ctok": maps["ctok"], "cslot": maps["cslot"]}
    else:  # the weighted gradient rows; the GEMMs read Phi, X and H in place through sel and ctok
        c = compact(p, G, Phi, alpha, tok, slot, sel=sel, keep=keep, mode=mode, out=b.get("compact"),
                    pack_phi=False, maps=maps, stream=stream)
        b.setdefault("compact", c)
    if mode == COMPACT_PHYSICAL:
        ctok, cslot = c["ctok"], c["cslot"]
        phi_rows = sel
        hc_rows = sel if p.swiglu else None
        x_rows = ctok if p.swiglu else None
    else:
        ctok, cslot = tok, slot
        phi_rows = hc_rows = None
        x_rows = tok if p.swiglu else None
    pmap = maps["pmap"] if maps is not None else None
    if overlap_scatter:
        if "side" not in b:
            b["side"] = torch.cuda.Stream(device=p.device)
            b["din_ready"] = torch.cuda.Event()
            b["side_ws"] = None if pmap is not None else torch.empty_like(p.workspace())
        if "out" not in b:
            nout = p.T if scatter_mode in (SCATTER_TOKEN, SCATTER_TOKEN_BESIDE) else p.T * p.K
            b["out"] = torch.empty(max(nout, 1), p.D if p.swiglu else p.F, dtype=torch.float32, device=p.device)
    if gathered and isinstance(H, Checkpoint):
        g = grouped_gemm_bwd_checkpoint(p, G, alpha, sel, ctok, PhiW, W2, X, H, W1, out=b.get("gemm"),
                                        din_ready=b["din_ready"] if overlap_scatter else None, stream=main)
    elif gathered:
        g = grouped_gemm_bwd_gathered(p, G, alpha, sel, ctok, PhiW, W2, X=X, H=H, W1=W1, out=b.get("gemm"),
                                      din_ready=b["din_ready"] if overlap_scatter else None, stream=main)
    else:
        g = grouped_gemm_bwd(p, c["Dlt"], Phi, W2, XC=X, HC=H, W1=W1, mode=mode, out=b.get("gemm"),
                             hc_rows=hc_rows, phi_rows=phi_rows, x_rows=x_rows,
                             din_ready=b["din_ready"] if overlap_scatter else None, stream=main)
    b.setdefault("gemm", g)
    if overlap_scatter:
        side = b["side"]
        side.wait_event(b["din_ready"])
        side_mode = SCATTER_TOKEN_BESIDE if scatter_mode == SCATTER_TOKEN else scatter_mode
        out = scatter(p, g["dIn"], ctok, cslot, n_rows=p.rows(mode), mode=side_mode, out=b["out"],
                      ws=b["side_ws"], pmap=pmap, stream=side)
        main.wait_stream(side)
    else:
        out = scatter(p, g["dIn"], ctok, cslot, n_rows=p.rows(mode), mode=scatter_mode, out=b.get("out"),
                      pmap=pmap, stream=main)
    b.setdefault("out", out)
    return {"R": b["R"], "sel": sel, "keep": keep, **c, **g, "out": out}


_MOST_COLUMNS, _MOST_PARTS = (1 << 31) - 8, (1 << 16) - 1  # of a part and of a row: the C calls count them in 32 bits


class Checkpoint:
    """Activation rows in 8 bits (the header's section on saved activations): codes ``q`` int8 [n, width] and ``scale``
    bf16 [n, parts, ceil(width / parts / 128)], one for every 128 columns of a part."""

    def __init__(self, q, scale):
        if q.dtype != torch.int8 or q.dim() != 2 or not q.is_contiguous():
            raise ValueError(f"q: expected contiguous int8 rows, got {q.dtype} of {tuple(q.shape)}")
        n, width = q.shape
        parts = scale.shape[1] if scale.dim() == 3 else 0
        if scale.dtype != torch.bfloat16 or not scale.is_contiguous() or parts < 1 or width % parts or (
                scale.shape != (n, parts, (width // parts + 127) // 128)):
            raise ValueError(f"scale: expected contiguous bfloat16 [rows, parts, groups of 128 columns], got "
                             f"{scale.dtype} of {tuple(scale.shape)} for q of {tuple(q.shape)}")
        if scale.get_device() != q.get_device():
            raise ValueError("q and scale must be on one device")
        if width // parts > _MOST_COLUMNS or parts > _MOST_PARTS:
            raise ValueError(f"q: {parts} parts of {width // parts} columns are more than the library counts")
        self.q, self.scale, self.parts, self.width = q, scale, parts, width // parts

    @classmethod
    def _of(cls, q, scale, parts, width):
        """Of tensors that need no checks (which take a third of a small call's host time)."""
        c = object.__new__(cls)
        c.q, c.scale, c.parts, c.width = q, scale, parts, width
        return c

    def _ptrs(self, name, n, parts, width, here):
        """Pointers of q and scale, if they hold at least n rows of that layout on the current device."""
        if self.q.shape[0] < n or (self.parts, self.width) != (parts, width) or self.q.get_device() != here:
            raise ValueError(f"{name}: expected a checkpoint of {n} rows of {parts} x {width} on the current device, got "
                             f"{self.q.shape[0]} of {self.parts} x {self.width} on {self.q.device}")
        return self.q.data_ptr(), self.scale.data_ptr()


def _new_checkpoint(n, parts, width, device, stream):
    q = _empty((n, parts * width), torch.int8, device, stream)
    return Checkpoint._of(q, _empty((n, parts, (width + 127) // 128), torch.bfloat16, device, stream), parts, width)


def checkpoint(rows, parts=1, out=None, stream=None):
    """``rows`` [n, width] (f32 or bf16) as a Checkpoint (lrmoe_checkpoint). ``parts``: equal column parts that share no
    scale (2 for [gate | up]). ``out``: a Checkpoint of that layout, overwritten."""
    here, dtype = torch._C._cuda_getDevice(), rows.dtype
    if (dtype is not torch.bfloat16 and dtype is not torch.float32) or rows.dim() != 2:
        raise ValueError("rows: expected f32 or bf16 [n, width]")
    (n, width), parts = rows.shape, int(parts)
    if parts < 1 or width % (8 * parts) or not width:
        raise ValueError("rows: the width must be a multiple of 8 in each part")
    width //= parts
    if width > _MOST_COLUMNS or parts > _MOST_PARTS:
        raise ValueError(f"rows: {parts} parts of {width} columns are more than the library counts")
    if rows.get_device() != here or not rows.is_contiguous():
        raise ValueError(f"rows: expected contiguous rows on the current device, got them on {rows.device}")
    raw = _stream(stream)
    if out is None:
        out = _new_checkpoint(n, parts, width, rows.device, stream)
        q, s = out.q.data_ptr(), out.scale.data_ptr()
    else:
        q, s = out._ptrs("out", n, parts, width, here)
    _lib.check(library().lrmoe_checkpoint(n, parts, width, BF16 if dtype is torch.bfloat16 else F32, rows.data_ptr(), q, s,
                                          raw), "lrmoe_checkpoint")
    return out


def restore(c: Checkpoint, dtype=torch.bfloat16, out=None, stream=None):
    """The rows that a Checkpoint stands for (lrmoe_restore), bf16 or f32 [n, width]."""
    here, q = torch._C._cuda_getDevice(), c.q
    shape = q.shape
    if out is not None:
        dtype = out.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError("dtype must be f32 or bf16")
    if q.get_device() != here:
        raise ValueError(f"c: expected a checkpoint on the current device, got it on {q.device}")
    raw = _stream(stream)
    if out is None:
        out = _empty(shape, dtype, q.device, stream)
        rows = out.data_ptr()
    else:
        rows = _want(out, "out", shape, dtype, here)
    _lib.check(library().lrmoe_restore(shape[0], c.parts, c.width, q.data_ptr(), c.scale.data_ptr(),
                                       BF16 if dtype is torch.bfloat16 else F32, rows, raw), "lrmoe_restore")
    return out


def expert_forward_checkpoint(p: Problem, X, tok, alpha, W1, W2, out=None, stream=None):
    """expert_forward that saves [gate | up] as a Checkpoint ("H") of the N pairs (lrmoe_expert_forward_checkpoint).
    "Phi" is what FC2 reads; a backward from the checkpoint does without it."""
    here, dt, o = torch._C._cuda_getDevice(), torch.bfloat16, out or {}
    n = max(p.N, 1)
    H = o.get("H") if o.get("H") is not None else _new_checkpoint(n, 2, p.F, p.device, stream)
    Phi = o.get("Phi") if o.get("Phi") is not None else _empty((n, p.F), dt, p.device, stream)
    Y = o.get("Y") if o.get("Y") is not None else _empty((n, p.D), dt, p.device, stream)
    q, s = H._ptrs("H", p.N, 2, p.F, here)
    _on_current(p, here)
    _lib.check(library().lrmoe_expert_forward_checkpoint(
        ctypes.byref(p.c), _ptr(p.seg_off_d), _ptr(X), _ptr(tok), _ptr(alpha), _ptr(W1), _ptr(W2), q, s, _ptr(Phi),
        _ptr(Y), _stream(stream)), "lrmoe_expert_forward_checkpoint")
    return {"H": Checkpoint._of(H.q[:p.N], H.scale[:p.N], 2, p.F), "Phi": Phi[:p.N], "Y": Y[:p.N]}


def _on_current(p, here):
    """The problem's arrays, workspace and the outputs allocated for it have to be on the current device."""
    if p.seg_off_d.get_device() != here:
        raise ValueError(f"the problem is on {p.seg_off_d.device}, which is not the current device")


def _saved(p, H, here):
    """Pointers of the pairs' saved rows in 8 bits: [gate | up], or Phi of FC2-only problems."""
    ptrs = H._ptrs("H", p.N, 2 if p.swiglu else 1, p.F, here)
    _on_current(p, here)
    return ptrs


def score_checkpoint(p: Problem, G, H: Checkpoint, alpha, tok, R=None, stream=None):
    """Step 1 from a Checkpoint of the pairs' [gate | up] rows (of their Phi rows, if FC2-only)."""
    q, s = _saved(p, H, torch._C._cuda_getDevice())
    if R is None:
        R = _empty((p.N,), torch.float32, p.device, stream)
    ws = p.workspace()
    _lib.check(library().lrmoe_score_checkpoint(ctypes.byref(p.c), _ptr(G), q, s, _ptr(alpha), _ptr(tok), _ptr(R),
                                                _ptr(ws), ws.numel(), _stream(stream)), "lrmoe_score_checkpoint")
    return R


def compact_checkpoint(p: Problem, sel, H: Checkpoint, alpha, out=None, stream=None):
    """compact_weighted from a Checkpoint: PhiW of the K_tot packed rows."""
    q, s = _saved(p, H, torch._C._cuda_getDevice())
    PhiW = out if out is not None else _empty((max(p.K_tot, 1), p.F), p.torch_dtype, p.device, stream)
    _lib.check(library().lrmoe_compact_checkpoint(ctypes.byref(p.c), _ptr(sel), q, s, _ptr(alpha), _ptr(PhiW),
                                                  _stream(stream)), "lrmoe_compact_checkpoint")
    return PhiW[:p.K_tot]


def grouped_gemm_bwd_checkpoint(p: Problem, G, alpha, sel, ctok, PhiW, W2, X, H: Checkpoint, W1, out=None,
                                accumulate=False, din_ready=None, stream=None):
    """grouped_gemm_bwd_gathered with [gate | up] from a Checkpoint (SwiGLU problems). X: rows of the storage dtype."""
    if not p.swiglu:
        raise ValueError("FC2-only problems have no [gate | up]: grouped_gemm_bwd_gathered")
    q, s = _saved(p, H, torch._C._cuda_getDevice())
    o = _gemm_outputs(p, p.K_tot, out)
    ws = p.workspace(COMPACT_PHYSICAL)
    _lib.check(library().lrmoe_grouped_gemm_bwd_checkpoint(
        ctypes.byref(p.c), _ptr(p.cseg_off_d), _ptr(G), _ptr(alpha), _ptr(sel), _ptr(ctok), _ptr(PhiW), _ptr(X), q, s,
        _ptr(W2), _ptr(W1), _ptr(o["dW2"]), _ptr(o["dW1"]), _ptr(o["dH"]), _ptr(o["dIn"]), int(bool(accumulate)),
        _ptr(ws), ws.numel(), _stream(stream), _event(din_ready, stream)), "lrmoe_grouped_gemm_bwd_checkpoint")
    return _gemm_results(p, p.K_tot, o)


class Router:
    """The router of one layer: T tokens, E experts of the whole layer, K slots per token, and the
    experts [first, first + local) that this GPU's pair lists cover (local=None: all from first).
    ``dtype``: F32 or BF16 logits. ``renorm``: a token's weights sum to ``scale``. ``device``:
    the one that is current when the calls are made.
    ``score``: "softmax" or "sigmoid" scores. ``groups``: the experts are that many equal runs, of which a token keeps
    the ``top_groups`` whose ``group_best`` (1 or 2) largest choice scores have the largest sum. A bias that
    enters the choice but not the weights is given to each ``route``."""

    def __init__(self, *, T, E, K, dtype=F32, first=0, local=None, renorm=False, scale=1.0, device="cuda",
                 score="softmax", groups=1, top_groups=1, group_best=1):
        self.T, self.E, self.K, self.dtype = int(T), int(E), int(K), int(dtype)
        self.first, self.local = int(first), int(E) - int(first) if local is None else int(local)
        self.renorm, self.scale = bool(renorm), float(scale)
        self.c = _lib.CRouter(T=self.T, E=self.E, K=self.K, first=self.first, local=self.local, dtype=self.dtype,
                              renorm=int(self.renorm), reserved=0, scale=self.scale)
        self.ref = ctypes.byref(self.c)
        if score not in _lib.SCORES:
            raise ValueError(f"unknown score {score!r}; expected one of {sorted(_lib.SCORES)}")
        self.score, self.groups, self.top_groups = score, int(groups), int(top_groups)
        self.group_best = int(group_best)
        self.scoring = _lib.CScoring(score=_lib.SCORES[score], groups=self.groups, top_groups=self.top_groups,
                                     group_best=self.group_best)
        self._scoring_ref = ctypes.byref(self.scoring)
        # softmax without groups: the calls without _scored, unless there is a bias
        self._plain = score == "softmax" and self.groups == self.top_groups == self.group_best == 1
        self.device = torch.device(device)
        self.torch_dtype = torch.bfloat16 if self.dtype == BF16 else torch.float32
        T, E, K, i32, f32 = self.T, self.E, self.K, torch.int32, torch.float32
        self._route_out = (("idx", (T, K), i32), ("w", (T, K), f32), ("counts", (E,), i32),
                           ("seg_off", (self.local + 1,), torch.int64), ("tok", (T * K,), i32),
                           ("slot", (T * K,), i32), ("alpha", (T * K,), f32), ("pmap", (T, K), i32))
        self._ws, self._ws_bytes, self._ws_size, self._streams = None, 0, {}, set()
        self._ws_captured, self._grown = False, []
        self.workspace_size()  # checks the router
        if not self._plain:
            _lib.check(library().lrmoe_scoring_check(self.ref, self._scoring_ref), "lrmoe_scoring_check")

    def workspace_size(self, n_seq=1) -> int:
        """lrmoe_router_workspace_size, asked once per number of sequences."""
        if n_seq not in self._ws_size:
            n = ctypes.c_size_t(0)
            _lib.check(library().lrmoe_router_workspace_size(self.ref, n_seq, ctypes.byref(n)),
                       "lrmoe_router_workspace_size")
            self._ws_size[n_seq] = int(n.value)
        return self._ws_size[n_seq]

    def workspace(self, n_seq=1, stream=None) -> torch.Tensor:
        """The router's scratch buffer. Calls that overlap on several streams, or graphs that
        may replay at the same time, need a Router each. A buffer that has become too small is
        kept if a call was captured with it: that graph may still use it, and needs the Router alive."""
        return self._scratch(n_seq, stream)[0]

    def _scratch(self, n_seq, stream):
        """(workspace, its bytes, raw handle of the stream)"""
        n, raw = self.workspace_size(n_seq), _stream(stream)
        if self._ws_bytes < n:
            if self._ws_captured:
                self._grown.append(self._ws)
            self._ws_captured = False
            self._ws, self._ws_bytes = _empty((n,), torch.uint8, self.device, stream), n
            self._ws_device = self._ws.get_device()
            self._streams.clear()
        if self._ws_device != torch._C._cuda_getDevice():  # the outputs allocated for it are there too
            raise ValueError(f"the router's workspace is on {self._ws.device}, which is not the current device")
        if raw and not self._ws_captured and _capturing(stream):  # the null stream, 0, is never captured
            self._ws_captured = True
        if raw not in self._streams:  # noted once per stream
            self._streams.add(raw)
            _used_on(stream, (self._ws,))
        return self._ws, self._ws_bytes, raw


def _capturing(stream):
    """Whether the current stream, or `stream`, records into a graph."""
    if torch.cuda.is_current_stream_capturing():
        return True
    if stream is None or stream.cuda_stream == _stream():
        return False
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _empty(shape, dtype, device, stream):
    """An output of a call on `stream` (None: the current one), allocated there: memory that other
    work of the current stream gave back is not written before that work is done."""
    # strides given save a third of torch.empty's host time
    strides = (1,) if len(shape) == 1 else (shape[1], 1) if len(shape) == 2 else (shape[1] * shape[2], shape[2], 1)
    if stream is None:
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)


def _used_on(stream, tensors):
    """Notes that work on `stream` uses `tensors`: memory that is freed meanwhile is given out again only behind
    that work."""
    if stream is None:
        stream = torch.cuda.current_stream()
    for t in tensors:
        t.record_stream(stream)


def _want(t, name, shape, dtype, here):
    """Pointer of a tensor after its shape, type and place (the current device) are checked
    (None -> NULL)."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or t.get_device() != here or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} of shape {tuple(shape)} on the current device, "
                         f"got {t.dtype} of {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _flags(t, name, n, here):
    """Pointer of a tensor of at least n zeros and ones (None -> NULL)."""
    if t is None:
        return None
    if t.dtype not in (torch.uint8, torch.bool) or t.numel() < n or t.get_device() != here:
        raise ValueError(f"{name}: expected {n} uint8 or bool entries on the current device")
    return _ptr(t)


def _outputs(given, wanted, device, here, stream):
    """(dict of outputs, their pointers): the given ones checked, the others allocated."""
    o = dict(given) if given else {}
    ptrs = []
    for name, shape, dt in wanted:
        t = o.get(name)
        if t is None:
            t = o[name] = _empty(shape, dt, device, stream)
            ptrs.append(t.data_ptr())
        else:
            ptrs.append(_want(t, name, shape, dt, here))
    return o, ptrs


def route(r: Router, logits, mask=None, out=None, stream=None, bias=None):
    """Top-K routing of ``logits`` [T, E] (lrmoe_route, lrmoe_route_scored): a dict of idx, w [T, K], counts [E],
    seg_off [local + 1] (device; ``.cpu()`` of it is Problem's seg_off), tok, slot, alpha [T*K] (rows
    at and after seg_off[local] are not written) and pmap [T, K]. ``mask`` [T] uint8 or bool: 0
    leaves a token out. ``bias`` f32 [E]: added to the scores in the choice, not in the weights. ``out``
    reuses buffers."""
    here = torch._C._cuda_getDevice()
    o, ptrs = _outputs(out, r._route_out, r.device, here, stream)
    ws, n, raw = r._scratch(1, stream)
    x, m = _want(logits, "logits", (r.T, r.E), r.torch_dtype, here), _flags(mask, "mask", r.T, here)
    if r._plain and bias is None:
        _lib.check(library().lrmoe_route(r.ref, x, m, *ptrs, ws.data_ptr(), n, raw), "lrmoe_route")
    else:
        _lib.check(library().lrmoe_route_scored(r.ref, r._scoring_ref, x,
                                                _want(bias, "bias", (r.E,), torch.float32, here), m, *ptrs,
                                                ws.data_ptr(), n, raw), "lrmoe_route_scored")
    return o


def bias_update(r: Router, bias, counts, rate, out=None, stream=None):
    """One step of the routing bias towards equal loads (lrmoe_bias_update): bias + rate * sign(mean(counts) - counts),
    f32 [E]. ``counts`` int32 [E]: route's, or their sum over the GPUs. ``out`` may be ``bias``."""
    here = torch._C._cuda_getDevice()
    if out is None:
        out = _empty((r.E,), torch.float32, r.device, stream)
    _lib.check(library().lrmoe_bias_update(r.ref, _want(counts, "counts", (r.E,), torch.int32, here), float(rate),
                                           _want(bias, "bias", (r.E,), torch.float32, here),
                                           _want(out, "out", (r.E,), torch.float32, here), _stream(stream)),
               "lrmoe_bias_update")
    return out


def _sequences(r, seq_off, here, stream):
    """(device offsets or None, number of sequences). Offsets on the host are checked and copied."""
    if seq_off is None:
        return None, 1
    if not isinstance(seq_off, torch.Tensor):
        seq_off = torch.as_tensor(seq_off, dtype=torch.int64)
    if seq_off.dtype != torch.int64 or seq_off.dim() != 1 or seq_off.numel() < 2:
        raise ValueError("seq_off must be int64 [n_seq + 1]")
    host = not seq_off.is_cuda
    if host:
        a = seq_off.tolist()
        if a[0] < 0 or a[-1] > r.T or any(x > y for x, y in zip(a, a[1:])):
            raise ValueError("seq_off must not decrease and stay inside [0, T]")
        seq_off = seq_off.to(r.device)
    if seq_off.get_device() != here:
        raise ValueError("seq_off must be on the current device, or on the host with the router on that device")
    if host and stream is not None:
        seq_off.record_stream(stream)
    return seq_off, seq_off.numel() - 1


def balance_loss(r: Router, logits, idx, coef=1.0, mask=None, seq_off=None, out=None, stream=None):
    """Per-expert counts and the balance loss of every sequence (lrmoe_balance_loss): a dict of loss
    [1], counts, psum [n_seq, E] and norm [n_seq]. ``seq_off`` (int64 [n_seq + 1], host or device;
    None: one sequence of all tokens): host offsets are checked and copied, which a capture into a
    graph does not allow. ``route_bwd`` takes the result as ``balance``."""
    here = torch._C._cuda_getDevice()
    off, S = _sequences(r, seq_off, here, stream)
    o, ptrs = _outputs(out, (("counts", (S, r.E), torch.int32), ("psum", (S, r.E), torch.float32),
                             ("norm", (S,), torch.float32), ("loss", (1,), torch.float32)), r.device, here, stream)
    ws, n, raw = r._scratch(S, stream)
    args = (_want(logits, "logits", (r.T, r.E), r.torch_dtype, here), _flags(mask, "mask", r.T, here),
            _want(idx, "idx", (r.T, r.K), torch.int32, here), _ptr(off), S, float(coef), *ptrs, ws.data_ptr(), n, raw)
    if r._plain:
        _lib.check(library().lrmoe_balance_loss(r.ref, *args), "lrmoe_balance_loss")
    else:
        _lib.check(library().lrmoe_balance_loss_scored(r.ref, r._scoring_ref, *args), "lrmoe_balance_loss_scored")
    return o


def route_bwd(r: Router, logits, idx, dalpha=None, pmap=None, balance=None, gloss=None, mask=None, seq_off=None,
              out=None, stream=None):
    """Gradient of the logits [T, E] (lrmoe_route_bwd). ``dalpha``: the routing weights' gradient, by
    pair row with ``pmap`` (alpha_grad's result and route's map), else [T, K]. ``balance``: what
    balance_loss returned for these logits, with the same ``seq_off`` and ``mask``; ``gloss`` (device
    f32 [1] or None = 1): the gradient of its loss. Either part may be None."""
    here = torch._C._cuda_getDevice()
    shape = (r.T, r.E)
    off, S = _sequences(r, seq_off, here, stream) if balance is not None else (None, 1)
    if out is None:
        out = _empty(shape, r.torch_dtype, r.device, stream)
    elif abs(out.data_ptr() - logits.data_ptr()) < r.T * r.E * logits.element_size():
        raise ValueError("out must not overlap the logits")
    n_pairs, d = 0, None
    if dalpha is not None:
        n_pairs = dalpha.numel()
        d = _want(dalpha, "dalpha", (n_pairs,) if pmap is not None else (r.T, r.K), torch.float32, here)
    counts = norm = None
    if balance is not None:
        counts = _want(balance["counts"], "counts", (S, r.E), torch.int32, here)
        norm = _want(balance["norm"], "norm", (S,), torch.float32, here)
    args = (_want(logits, "logits", shape, r.torch_dtype, here), _flags(mask, "mask", r.T, here),
            _want(idx, "idx", (r.T, r.K), torch.int32, here), d, _want(pmap, "pmap", (r.T, r.K), torch.int32, here),
            n_pairs, _ptr(off), S, counts, norm, _want(gloss, "gloss", (1,), torch.float32, here),
            _want(out, "out", shape, r.torch_dtype, here), _stream(stream))
    if r._plain:
        _lib.check(library().lrmoe_route_bwd(r.ref, *args), "lrmoe_route_bwd")
    else:
        _lib.check(library().lrmoe_route_bwd_scored(r.ref, r._scoring_ref, *args), "lrmoe_route_bwd_scored")
    return out


def alpha_grad(p: Problem, G, Y, alpha, pmap, keep=None, out=None, stream=None):
    """Gradient of the N pairs' routing weights from expert_forward's rows Y and the output's
    gradient G (lrmoe_alpha_grad); ``pmap`` [T, K] from route, ``keep`` [N] uint8 from select."""
    here, f32, dt, N = torch._C._cuda_getDevice(), torch.float32, p.torch_dtype, p.N
    if out is None:
        out = _empty((N,), f32, p.device, stream)
    if alpha.dtype != f32 or out.dtype != f32 or alpha.numel() < N or out.numel() < N:
        raise ValueError("alpha and out: expected f32 of at least N elements")
    if G.dtype != dt or Y.dtype != dt or G.dim() != 2 or Y.dim() != 2 or G.shape[1] != p.D or Y.shape[1] != p.D or (
            G.shape[0] < p.T or Y.shape[0] < N):
        raise ValueError(f"G and Y: expected {dt} of T and N rows of {p.D}")
    if not alpha.get_device() == out.get_device() == G.get_device() == Y.get_device() == here:
        raise ValueError("alpha, out, G and Y must be on the current device")
    _lib.check(library().lrmoe_alpha_grad(ctypes.byref(p.c), _ptr(G), _ptr(Y), _ptr(alpha),
                                          _want(pmap, "pmap", (p.T, p.K), torch.int32, here),
                                          _flags(keep, "keep", N, here), _ptr(out), _stream(stream)),
               "lrmoe_alpha_grad")
    return out


class AdamW:
    """AdamW over a list of tensors, updated in place by one call (lrmoe_adamw).

    ``weights``: f32 or bf16 tensors, all of one type; ``masters``: their f32 masters (bf16 weights
    only), or None; ``grads``: the gradient buffers the backward writes (f32 or bf16, all of one
    type), if they are the same at every step. Others are given to each ``step``: new ones are checked
    one by one (about 1 us of host time each), and more than 48 tensors then take a launch for every
    48 instead of one. ``bits``: 32 or 8 bits of state per moment. The
    states ``m``, ``v`` (8 bits: e4m3 codes, v's of its square root, with ``m_scale``, ``v_scale`` per 256
    elements) start at zero unless given. ``first``: 8 bits, the counter of each tensor's first
    element for the random rounding (multiples of 256; None: one tensor behind the other).
    ``t`` counts the steps taken. Buffers must not overlap; gradients, which are only read, may share one."""

    def __init__(self, weights, grads=None, masters=None, m=None, v=None, m_scale=None, v_scale=None, *, lr=1e-3,
                 betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, bits=32, first=None, step=0, seed=0):
        self.w, self.masters = list(weights), None if masters is None else list(masters)
        if not self.w:
            raise ValueError("AdamW needs at least one tensor")
        dev = self.w[0].device
        sizes = [t.numel() for t in self.w]
        if bits not in (32, 8):
            raise ValueError("bits must be 32 or 8")
        st = torch.float8_e4m3fn if bits == 8 else torch.float32

        self._own = []  # what is allocated here; the caller looks after the rest

        def states(given, dt, n, fill=0):
            if given is not None:
                return list(given)
            new = [torch.full((k,), fill, dtype=torch.uint8 if dt == torch.float8_e4m3fn else dt,
                              device=dev).view(dt) for k in n]
            self._own += new
            return new

        blocks = [(k + 255) // 256 for k in sizes]
        self.m, self.v = states(m, st, sizes), states(v, st, sizes)
        self.m_scale = states(m_scale, torch.float32, blocks, 1) if bits == 8 else None
        self.v_scale = states(v_scale, torch.float32, blocks, 1) if bits == 8 else None
        at = 0
        if first is None:
            first = []
            for b in blocks:
                first.append(at)
                at += b * 256
        self.t, self.lr, self.weight_decay = int(step), lr, weight_decay
        wt = self.w[0].dtype
        if wt not in (torch.float32, torch.bfloat16):
            raise ValueError("weights must be f32 or bf16")
        for name, ts, dt, n in (("weights", self.w, wt, sizes), ("masters", self.masters, torch.float32, sizes),
                                ("m", self.m, st, sizes), ("v", self.v, st, sizes),
                                ("m_scale", self.m_scale, torch.float32, blocks),
                                ("v_scale", self.v_scale, torch.float32, blocks)):
            if ts is not None and (len(ts) != len(sizes) or any(
                    t.dtype != dt or t.numel() != k or t.device != dev for t, k in zip(ts, n))):
                raise ValueError(f"{name}: one tensor of {dt} per weight, of its size, on {dev}")
        if len(first) != len(sizes):
            raise ValueError("first: one counter per weight")
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())
                       for ts in (self.w, self.masters, self.m, self.v, self.m_scale, self.v_scale)
                       if ts is not None for t in ts if t.numel())
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise ValueError("AdamW's buffers overlap")
        self._sizes, self._starts, self._ends = sizes, [a for a, _ in spans], [b for _, b in spans]
        self.c = _lib.CAdamwConfig(w_dtype=BF16 if wt == torch.bfloat16 else F32, grad_dtype=F32,
                                   master=int(masters is not None), state_bits=bits, lr=lr, beta1=betas[0],
                                   beta2=betas[1], eps=eps, weight_decay=weight_decay, grad_scale=1.0, step=1,
                                   seed=int(seed), reserved=0)
        self._table = (_lib.CAdamwTensor * len(sizes))()
        for i, k in enumerate(sizes):
            e = self._table[i]
            e.w, e.master = _ptr(self.w[i]), _ptr(self.masters[i]) if masters is not None else None
            e.m, e.v, e.n, e.first = _ptr(self.m[i]), _ptr(self.v[i]), k, int(first[i])
            if bits == 8:
                e.m_scale, e.v_scale = _ptr(self.m_scale[i]), _ptr(self.v_scale[i])
        words = np.frombuffer(self._table, np.uint64).reshape(len(sizes), -1)  # the table's fields are 8 bytes each
        self._table_grads = words[:, _lib.CAdamwTensor.grad.offset // 8]
        self._scalars = self._plan = None
        self._captured, self._plans, self._noted = [], 0, {}
        self.grads = None
        if grads is not None:
            self.bind(grads)
        _lib.check(library().lrmoe_adamw_step_scalars(ctypes.byref(self.c), ctypes.byref(_lib.CAdamwScalars())),
                   "lrmoe_adamw_step_scalars")

    def bind(self, grads):
        """Takes these tensors as the gradient buffers from now on."""
        grads = list(grads)
        dt, dev = grads[0].dtype if grads else None, self.w[0].device
        if len(grads) != len(self.w) or dt not in (torch.float32, torch.bfloat16) or any(
                g.dtype != dt or g.numel() != n or g.device != dev for g, n in zip(grads, self._sizes)):
            raise ValueError("grads: one f32 or bf16 tensor per weight, of its size, all of one type")
        ptrs = [_ptr(g) for g in grads]  # all of them first: a tensor that is refused leaves the old ones bound
        size = grads[0].element_size()
        for at, n in zip(ptrs, self._sizes):
            i = bisect.bisect_left(self._starts, at + n * size) - 1  # the last buffer that starts before its end
            if n and i >= 0 and self._ends[i] > at:
                raise ValueError("grads: a gradient overlaps the weights, their masters or the states")
        self._table_grads[:] = ptrs
        self.c.grad_dtype = BF16 if dt == torch.bfloat16 else F32
        self.grads, self._plan = grads, None

    def _plan_ptr(self, stream):
        """The plan in device memory for more tensors than one launch's arguments take. It is made at
        the second step with the same gradient buffers: a copy of it to the device would cost a
        program that binds new ones at every step more than the launches it saves."""
        if len(self.w) <= 48:
            return None
        if self._plan is None:
            self._plan = False
        elif self._plan is False and not _capturing(stream):
            n, lib = ctypes.c_size_t(0), library()
            args = (self._table, len(self.w), ctypes.byref(self.c))
            _lib.check(lib.lrmoe_adamw_plan(*args, None, ctypes.byref(n)), "lrmoe_adamw_plan")
            host = torch.empty(n.value, dtype=torch.uint8)
            _lib.check(lib.lrmoe_adamw_plan(*args, host.data_ptr(), ctypes.byref(n)), "lrmoe_adamw_plan")
            self._plan = host.to(self.w[0].device)
            self._plans += 1
        return self._plan.data_ptr() if self._plan is not False else None

    def _used_on(self, stream):
        """Raw handle of `stream`, on which work uses what this object allocated."""
        raw = _stream(stream)
        now = self._plans, self._scalars is not None
        seen = self._noted.get(raw)
        if seen != now:  # noted once per stream
            own = [] if seen else list(self._own)
            if isinstance(self._plan, torch.Tensor) and (not seen or seen[0] != now[0]):
                own.append(self._plan)
            if now[1] and not (seen and seen[1]):
                own.append(self._scalars)
            _used_on(stream, own)
            self._noted[raw] = now
        return raw

    def _config(self, grad_scale):
        self.c.step, self.c.lr, self.c.weight_decay, self.c.grad_scale = self.t, self.lr, self.weight_decay, grad_scale

    def _check_place(self):
        if self.w[0].get_device() != torch.cuda.current_device():
            raise ValueError("AdamW's tensors must be on the current device")

    def step(self, grads=None, grad_scale=1.0, stream=None):
        """One step. Inside a captured graph call ``step_captured`` instead."""
        if grads is not None:
            self.bind(grads)
        if self.grads is None:
            raise ValueError("AdamW has no gradient buffers: pass grads")
        self._check_place()
        if _capturing(stream):
            raise ValueError("a graph would repeat this very step: capture step_captured")
        self.t += 1
        try:
            self._config(grad_scale)
            plan = self._plan_ptr(stream)
            _lib.check(library().lrmoe_adamw(self._table, len(self.w), ctypes.byref(self.c), plan, None,
                                             self._used_on(stream)), "lrmoe_adamw")
        except Exception:
            self.t -= 1
            raise

    def advance(self, grad_scale=1.0, stream=None):
        """Counts one step and copies its scalars (step, lr, weight_decay, grad_scale) to the device, on
        `stream` (None: the current one), without waiting for it. Call it before each replay of a graph
        that holds ``step_captured``, on the stream of the replays: the copy then follows those before
        it, which read their own step's scalars from the same place."""
        gpu = self.w[0].is_cuda
        if gpu:
            self._check_place()
            if _capturing(stream):
                raise ValueError("advance belongs before a replay, not into the graph")
        host = _lib.CAdamwScalars()
        self.t += 1
        try:
            self._config(grad_scale)
            _lib.check(library().lrmoe_adamw_step_scalars(ctypes.byref(self.c), ctypes.byref(host)),
                       "lrmoe_adamw_step_scalars")
            values = torch.frombuffer(bytearray(host), dtype=torch.int32)
            if self._scalars is None:
                self._scalars = _empty((8,), torch.int32, self.w[0].device, stream)
            if gpu:
                self._used_on(stream)
                values = values.pin_memory()  # torch gives it out again only behind the copy
            with torch.cuda.stream(stream):
                self._scalars.copy_(values, non_blocking=True)
        except Exception:
            self.t -= 1
            raise

    def step_captured(self, stream=None):
        """The update with the scalars of the last ``advance``, for capture into a graph. What a graph
        reads stays alive with this object: the plan and the gradient buffers bound now."""
        if self._scalars is None or self.grads is None:
            raise ValueError("call advance (and bind the gradient buffers) before step_captured")
        self._check_place()
        plan = self._plan_ptr(stream)
        if _capturing(stream):
            self._captured.append((self._plan, self.grads))
        _lib.check(library().lrmoe_adamw(self._table, len(self.w), ctypes.byref(self.c), plan,
                                         _ptr(self._scalars), self._used_on(stream)), "lrmoe_adamw")
