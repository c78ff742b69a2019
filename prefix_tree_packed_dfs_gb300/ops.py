"""Torch-facing wrappers over the C ABI (same names as ``include/tpk.h``).

PyTorch only provides device memory and the current stream; the wrappers check
dtypes/shapes/contiguity, allocate outputs with torch and pass raw pointers.
"""
import ctypes
import math

import numpy as np
import torch

from . import binding as B


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _need(t, dtype, name, ndim=None, cuda=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if cuda and not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (no CPU path exists)" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if ndim is not None and t.dim() != ndim:
        raise ValueError("%s must have %d dims" % (name, ndim))


class Plan:
    """Host packing plan (``tpk_plan_build``)."""

    def __init__(self, tokens, seq_offsets, trained=None, group_ids=None, row_capacity=65536,
                 min_shared=64, placement="bfd"):
        lib = B.load()
        self._lib = lib
        self._h = None
        tokens = np.ascontiguousarray(tokens, dtype=np.int32)
        offs = np.ascontiguousarray(seq_offsets, dtype=np.int64)
        n = len(offs) - 1
        tr = None if trained is None else np.ascontiguousarray(trained, dtype=np.uint8)
        gr = None if group_ids is None else np.ascontiguousarray(group_ids, dtype=np.int32)
        if tr is not None and len(tr) != len(tokens):
            raise ValueError("trained must have one flag per token")
        if gr is not None and len(gr) != n:
            raise ValueError("group_ids must have one id per sequence")
        opts = B.PlanOpts(int(row_capacity), int(min_shared),
                          {"bfd": B.PLACE_BFD, "next_fit": B.PLACE_NEXT_FIT, "groups": B.PLACE_GROUPS}[placement])
        h = ctypes.c_void_p()
        st = lib.tpk_plan_build(tokens.ctypes.data, offs.ctypes.data, n,
                                None if tr is None else tr.ctypes.data,
                                None if gr is None else gr.ctypes.data,
                                ctypes.byref(opts), ctypes.byref(h))
        B.check(st, "tpk_plan_build")
        self._h = h
        info = B.PlanInfo()
        B.check(lib.tpk_plan_info_get(h, ctypes.byref(info)), "tpk_plan_info_get")
        self.info = info.as_dict()

    @classmethod
    def from_sequences(cls, sequences, trained=None, **kw):
        seqs = [np.asarray(s) for s in sequences]
        offs = np.zeros(len(seqs) + 1, dtype=np.int64)
        offs[1:] = np.cumsum([len(s) for s in seqs])
        tr = None if trained is None else np.concatenate([np.asarray(t) for t in trained])
        return cls(np.concatenate(seqs), offs, trained=tr, **kw)

    @property
    def handle(self):
        return self._h

    def __getattr__(self, name):
        info = self.__dict__.get("info")
        if info is not None and name in info:
            return info[name]
        raise AttributeError(name)

    def export(self):
        i = self.info
        F, R, n, rows = i["n_fwd"], i["n_raw"], i["n_seqs"], i["n_rows"]
        out = {
            "row_offsets": np.zeros(rows + 1, np.int64), "row_loads": np.zeros(rows, np.int64),
            "row_of_seq": np.zeros(n, np.int32), "fwd_token": np.zeros(F, np.int32),
            "fwd_src": np.zeros(F, np.int32), "parent": np.zeros(F, np.int32), "depth": np.zeros(F, np.int32),
            "token_index": np.zeros(R, np.int32), "subtree_end": np.zeros(F, np.int32),
        }
        order = ["row_offsets", "row_loads", "row_of_seq", "fwd_token", "fwd_src", "parent", "depth",
                 "token_index", "subtree_end"]
        B.check(self._lib.tpk_plan_export(self._h, *[out[k].ctypes.data for k in order]), "tpk_plan_export")
        return out

    def worklists(self):
        i = self.info
        T, NB, KT, NQB = i["n_qtiles"], i["n_kblocks"], i["n_ktiles"], i["n_qblocks"]
        out = {
            "qt_q0": np.zeros(T, np.int32), "qt_nq": np.zeros(T, np.int32), "qt_kb_begin": np.zeros(T + 1, np.int32),
            "kb": np.zeros(2 * NB, np.int32), "qt_order": np.zeros(T, np.int32),
            "kt_k0": np.zeros(KT, np.int32), "kt_nk": np.zeros(KT, np.int32),
            "kt_qb_begin": np.zeros(KT + 1, np.int32), "qb": np.zeros(2 * NQB, np.int32),
            "kt_order": np.zeros(KT, np.int32),
        }
        order = ["qt_q0", "qt_nq", "qt_kb_begin", "kb", "qt_order", "kt_k0", "kt_nk", "kt_qb_begin", "qb",
                 "kt_order"]
        B.check(self._lib.tpk_plan_worklists(self._h, *[out[k].ctypes.data for k in order]), "tpk_plan_worklists")
        return out

    def raw_of_forwarded(self):
        """(fwd_raw_begin [F+1], fwd_raw [R]): the raw tokens of each forwarded position, ascending."""
        F, R = self.info["n_fwd"], self.info["n_raw"]
        begin, raw = np.zeros(F + 1, np.int32), np.zeros(R, np.int32)
        B.check(self._lib.tpk_plan_raw_of_forwarded(self._h, begin.ctypes.data, raw.ctypes.data),
                "tpk_plan_raw_of_forwarded")
        return begin, raw

    def segments(self):
        """Segment instances by tree level: (level_begin [n_levels+1],
        seg_start, seg_len, seg_parent [n_instances]), int32."""
        n, L = self.info["n_seg_instances"], self.info["n_seg_levels"]
        out = (np.zeros(L + 1, np.int32), np.zeros(n, np.int32), np.zeros(n, np.int32), np.zeros(n, np.int32))
        B.check(self._lib.tpk_plan_segments(self._h, *[a.ctypes.data for a in out]), "tpk_plan_segments")
        return out

    def shard_rows(self, world):
        """Whole rows to `world` data-parallel ranks, heaviest row first to the
        least-loaded rank (work = useful pairs).  Returns (rank_of_row int32
        [n_rows], rank_pairs int64 [world])."""
        rows = self.info["n_rows"]
        rank_of_row, rank_pairs = np.zeros(rows, np.int32), np.zeros(world, np.int64)
        B.check(self._lib.tpk_plan_shard_rows(self._h, int(world), rank_of_row.ctypes.data, rank_pairs.ctypes.data),
                "tpk_plan_shard_rows")
        return rank_of_row, rank_pairs

    def sequences_of_rank(self, rank_of_row, rank):
        """Indices (input order) of the sequences whose row `rank` owns."""
        return np.flatnonzero(np.asarray(rank_of_row)[self.export()["row_of_seq"]] == rank)

    def rank_plan(self, sequences, rank_of_row, rank, row_capacity, min_shared=64, trained=None):
        """The plan of rank `rank`'s rows (``shard_rows``): its sequences,
        planned with their row in this plan as the group and one row per
        group, i.e. exactly those rows.  Returns (plan, sequence indices);
        ``sequences`` / ``trained`` are the inputs this plan was built from."""
        idx = self.sequences_of_rank(rank_of_row, rank)
        rows = self.export()["row_of_seq"][idx]
        sub = Plan.from_sequences([sequences[i] for i in idx],
                                  trained=None if trained is None else [trained[i] for i in idx],
                                  group_ids=rows, row_capacity=row_capacity, min_shared=min_shared,
                                  placement="groups")
        return sub, idx

    def device_bytes(self):
        return int(self._lib.tpk_plan_device_bytes(self._h))

    def field_offset(self, field):
        off = ctypes.c_size_t()
        B.check(self._lib.tpk_plan_field_offset(self._h, field, ctypes.byref(off)), "tpk_plan_field_offset")
        return off.value

    def to_device(self, device="cuda"):
        return DevicePlan(self, device)

    def close(self):
        if self._h is not None:
            self._lib.tpk_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class DevicePlan:
    """A plan plus its device image (one torch uint8 buffer)."""

    def __init__(self, plan, device="cuda"):
        self.plan = plan
        nbytes = max(plan.device_bytes(), 256)
        self.image = torch.empty(nbytes, dtype=torch.uint8, device=device)
        if self.image.data_ptr() % 256:
            raise RuntimeError("device image not 256-byte aligned")
        B.check(plan._lib.tpk_plan_upload(plan.handle, _ptr(self.image), _stream()), "tpk_plan_upload")
        F, R = plan.info["n_fwd"], plan.info["n_raw"]
        self.depth = self._field(B.FIELD_DEPTH, F)
        self.token_index = self._field(B.FIELD_TOKEN_INDEX, R)
        self.subtree_end = self._field(B.FIELD_SUBTREE_END, F)
        self.parent = self._field(B.FIELD_PARENT, F)
        self.fwd_raw_begin = self._field(B.FIELD_FWD_RAW_BEGIN, F + 1)
        self.fwd_raw = self._field(B.FIELD_FWD_RAW, R)
        n_inst = plan.info["n_seg_instances"]
        self.seg_start = self._field(B.FIELD_SEG_START, n_inst)
        self.seg_len = self._field(B.FIELD_SEG_LEN, n_inst)
        self.seg_parent = self._field(B.FIELD_SEG_PARENT, n_inst)
        self.seg_off = self._field(B.FIELD_SEG_OFF, n_inst)

    def _field(self, field, n):
        off = self.plan.field_offset(field)
        return self.image[off:off + 4 * n].view(torch.int32)

    @property
    def n_fwd(self):
        return self.plan.info["n_fwd"]

    @property
    def n_raw(self):
        return self.plan.info["n_raw"]


def rope_by_depth(q, k, depth, base, inverse=False, q_out=None, k_out=None):
    """RoPE of q [F,Hq,d] and/or k [F,Hkv,d] at ``depth`` (int32 [F]).

    In place unless ``q_out`` / ``k_out`` are given.  Returns (q_out, k_out)."""
    lib = B.load()
    ref = q if q is not None else k
    F, _, d = ref.shape
    if q is not None:
        _need(q, torch.bfloat16, "q", 3)
        q_out = q if q_out is None else q_out
        _need(q_out, torch.bfloat16, "q_out", 3)
    if k is not None:
        _need(k, torch.bfloat16, "k", 3)
        k_out = k if k_out is None else k_out
        _need(k_out, torch.bfloat16, "k_out", 3)
    _need(depth, torch.int32, "depth", 1)
    if depth.numel() != F or (q is not None and k is not None and k.shape[0] != F):
        raise ValueError("shape mismatch")
    Hq = q.shape[1] if q is not None else 0
    Hkv = k.shape[1] if k is not None else 0
    B.check(lib.tpk_rope_by_depth(_ptr(q), _ptr(k), _ptr(q_out) if q is not None else None,
                                  _ptr(k_out) if k is not None else None, _ptr(depth), F, Hq, Hkv, d,
                                  float(base), 1 if inverse else 0, _stream()), "tpk_rope_by_depth")
    return q_out, k_out


def _shape(t, shape, name):
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _on_device(ref, *named):
    """Every tensor (None skipped) a CUDA tensor on ref's device.  Checked after
    the shapes, so a wrong shape is reported as such wherever the tensors live."""
    for t, n in ((ref, "q"),) + named:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("%s must be a CUDA tensor (no CPU path exists)" % n)
        if t.device != ref.device:
            raise ValueError("%s is on %s, expected %s" % (n, t.device, ref.device))


def _attn_shapes(dplan, q, k, v):
    """(F, Hq, Hkv, d) of q [F,Hq,d], k/v [F,Hkv,d], checked against the plan."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, n, 3, cuda=False)
    F, Hq, d = q.shape
    Hkv = k.shape[1]
    if F != dplan.n_fwd:
        raise ValueError("q has %d rows, the plan has %d forwarded positions" % (F, dplan.n_fwd))
    _shape(k, (F, Hkv, d), "k")
    _shape(v, (F, Hkv, d), "v")
    return F, Hq, Hkv, d


def _opts(precise, rope_base=None, o_lo=None):
    return B.AttnOpts(B.PREC_PRECISE if precise else B.PREC_FAST, 0,
                      0.0 if rope_base is None else float(rope_base), None if o_lo is None else o_lo.data_ptr())


def tree_attn_fwd(dplan, q, k, v, scale=None, out=None, lse=None, dev_err=None, precise=False, o_lo=None):
    """Forward tree attention; returns (O [F,Hq,d] bf16, LSE [Hq,F] fp32).

    ``precise``: P enters the PV product as a hi + lo bf16 pair, and O's bf16
    rounding residual is written to ``o_lo`` (allocated if None); the return
    value is then (O, LSE, O_lo)."""
    lib = B.load()
    F, Hq, Hkv, d = _attn_shapes(dplan, q, k, v)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((Hq, F), dtype=torch.float32, device=q.device)
    _need(out, torch.bfloat16, "out", 3, cuda=False)
    _shape(out, (F, Hq, d), "out")
    _need(lse, torch.float32, "lse", 2, cuda=False)
    _shape(lse, (Hq, F), "lse")
    if precise:
        o_lo = torch.empty_like(q) if o_lo is None else o_lo
        _need(o_lo, torch.bfloat16, "o_lo", 3, cuda=False)
        _shape(o_lo, (F, Hq, d), "o_lo")
    if dev_err is not None:
        _need(dev_err, torch.int32, "dev_err", cuda=False)
    _on_device(q, (k, "k"), (v, "v"), (dplan.image, "the plan image"), (out, "out"), (lse, "lse"),
               (o_lo if precise else None, "o_lo"), (dev_err, "dev_err"))
    opts = _opts(precise, None, o_lo if precise else None)
    st = lib.tpk_tree_attn_fwd_ex(dplan.plan.handle, _ptr(dplan.image), _ptr(q), _ptr(k), _ptr(v), _ptr(out),
                                  _ptr(lse), Hq, Hkv, d, scale, ctypes.byref(opts), _ptr(dev_err), _stream())
    B.check(st, "tpk_tree_attn_fwd_ex")
    return (out, lse, o_lo) if precise else (out, lse)


def attn_workspace_bytes(dplan, Hq, Hkv, d, backward):
    lib = B.load()
    return int(lib.tpk_attn_workspace_bytes(dplan.plan.handle, Hq, Hkv, d, 1 if backward else 0))


def tree_attn_bwd(dplan, q, k, v, o, lse, do, scale=None, dq=None, dk=None, dv=None, workspace=None,
                  dev_err=None, phases=(0, 1, 2), precise=False, o_lo=None, rope_base=None):
    """Backward tree attention; returns (dQ, dK, dV).

    Gradients are w.r.t. the rotated q, k unless ``rope_base`` is given, in
    which case the inverse RoPE at depth is applied inside the kernels and
    dQ, dK are w.r.t. the un-rotated inputs.  ``precise`` selects the hi + lo
    bf16 products (and uses the forward's ``o_lo`` for dO . O when given).
    ``phases`` selects the launches (0 prep, 1 dK/dV pass, 2 dQ pass); the
    default runs all three in order."""
    lib = B.load()
    F, Hq, Hkv, d = _attn_shapes(dplan, q, k, v)
    for t, n in ((o, "o"), (do, "do")):
        _need(t, torch.bfloat16, n, 3, cuda=False)
        _shape(t, (F, Hq, d), n)
    _need(lse, torch.float32, "lse", 2, cuda=False)
    _shape(lse, (Hq, F), "lse")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for t, n, shp in ((dq, "dq", (F, Hq, d)), (dk, "dk", (F, Hkv, d)), (dv, "dv", (F, Hkv, d))):
        _need(t, torch.bfloat16, n, 3, cuda=False)
        _shape(t, shp, n)
    if o_lo is not None:
        _need(o_lo, torch.bfloat16, "o_lo", 3, cuda=False)
        _shape(o_lo, (F, Hq, d), "o_lo")
    need = attn_workspace_bytes(dplan, Hq, Hkv, d, True)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor")
    ws_bytes = workspace.numel() * workspace.element_size()
    if ws_bytes < need:
        raise ValueError("workspace has %d bytes, the backward needs %d" % (ws_bytes, need))
    if dev_err is not None:
        _need(dev_err, torch.int32, "dev_err", cuda=False)
    _on_device(q, (k, "k"), (v, "v"), (dplan.image, "the plan image"), (o, "o"), (do, "do"), (lse, "lse"),
               (dq, "dq"), (dk, "dk"), (dv, "dv"), (o_lo, "o_lo"), (workspace, "workspace"), (dev_err, "dev_err"))
    opts = _opts(precise, rope_base, o_lo)
    args = (dplan.plan.handle, _ptr(dplan.image), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do),
            _ptr(dq), _ptr(dk), _ptr(dv), Hq, Hkv, d, scale, ctypes.byref(opts), _ptr(workspace), ws_bytes,
            _ptr(dev_err), _stream())
    if tuple(phases) == (0, 1, 2):
        B.check(lib.tpk_tree_attn_bwd_ex(B.BWD_ALL, *args), "tpk_tree_attn_bwd_ex")
    else:
        for ph in phases:
            B.check(lib.tpk_tree_attn_bwd_ex(int(ph), *args), "tpk_tree_attn_bwd_ex")
    return dq, dk, dv


def scatter_token_index(token_index, src=None, lse_src=None, dst=None, lse_dst=None):
    """Raw-order copies: dst[r] = src[token_index[r]], lse_dst[:, r] = lse_src[:, token_index[r]]."""
    lib = B.load()
    _need(token_index, torch.int32, "token_index", 1)
    R = token_index.numel()
    if src is not None:
        _need(src, torch.bfloat16, "src", 3)
        F, H, d = src.shape
        if dst is None:
            dst = torch.empty((R, H, d), dtype=src.dtype, device=src.device)
    if lse_src is not None:
        _need(lse_src, torch.float32, "lse_src", 2)
        H, F = lse_src.shape
        if lse_dst is None:
            lse_dst = torch.empty((H, R), dtype=torch.float32, device=lse_src.device)
    if src is None and lse_src is None:
        return None, None
    d = src.shape[2] if src is not None else 8
    B.check(lib.tpk_scatter_token_index(_ptr(token_index), R, F, _ptr(src), _ptr(dst), _ptr(lse_src),
                                        _ptr(lse_dst), H, d, _stream()), "tpk_scatter_token_index")
    return dst, lse_dst


def gather_to_forwarded(dplan, src, dst=None):
    """Packed-layout copy of a per-raw-token payload: dst[f] = src[owner of f].

    ``src`` is any contiguous device tensor whose first dimension is the raw
    token (R); every forwarded position takes its owner's row (the lowest
    raw token mapping to it)."""
    lib = B.load()
    R, F = dplan.n_raw, dplan.n_fwd
    if not src.is_cuda or not src.is_contiguous() or src.shape[0] != R:
        raise ValueError("src must be a contiguous device tensor with %d rows" % R)
    if dst is None:
        dst = torch.empty((F,) + tuple(src.shape[1:]), dtype=src.dtype, device=src.device)
    if dst.dtype != src.dtype or tuple(dst.shape) != (F,) + tuple(src.shape[1:]) or not dst.is_contiguous():
        raise ValueError("dst must be a contiguous %s tensor of shape %s" % (src.dtype, (F,) + tuple(src.shape[1:])))
    row_bytes = src[0].numel() * src.element_size() if R else 1
    B.check(lib.tpk_gather_to_forwarded(_ptr(dplan.fwd_raw_begin), _ptr(dplan.fwd_raw), F, R, _ptr(src), _ptr(dst),
                                        row_bytes, _stream()), "tpk_gather_to_forwarded")
    return dst


def sum_to_forwarded(dplan, src=None, lse_src=None, dst=None, lse_dst=None):
    """Adjoint of the raw-order scatter: dst[f] = sum of src[r] over the raw tokens r of f.

    ``src`` [R, H, d] bf16 -> [F, H, d] bf16; ``lse_src`` [H, R] fp32 -> [H, F]
    (a per-token fp32 weight is the case H = 1).  fp32 sums in ascending raw
    order."""
    lib = B.load()
    R, F = dplan.n_raw, dplan.n_fwd
    H, d = 1, 8
    if src is not None:
        _need(src, torch.bfloat16, "src", 3)
        if src.shape[0] != R:
            raise ValueError("src must have %d rows" % R)
        _, H, d = src.shape
        if dst is None:
            dst = torch.empty((F, H, d), dtype=src.dtype, device=src.device)
    if lse_src is not None:
        _need(lse_src, torch.float32, "lse_src", 2)
        if lse_src.shape[1] != R or (src is not None and lse_src.shape[0] != H):
            raise ValueError("lse_src must be [H, %d]" % R)
        H = lse_src.shape[0]
        if lse_dst is None:
            lse_dst = torch.empty((H, F), dtype=torch.float32, device=lse_src.device)
    if src is None and lse_src is None:
        return None, None
    B.check(lib.tpk_sum_to_forwarded(_ptr(dplan.fwd_raw_begin), _ptr(dplan.fwd_raw), F, R, _ptr(src), _ptr(dst),
                                     _ptr(lse_src), _ptr(lse_dst), H, d, _stream()), "tpk_sum_to_forwarded")
    return dst, lse_dst


def gdn_conv(dplan, x, w, y=None):
    """Causal depthwise convolution + SiLU along each position's path
    (``tpk_gdn_conv``): x [F, C] bf16, w [C, W] fp32 -> y [F, C] bf16."""
    lib = B.load()
    _need(x, torch.bfloat16, "x", 2, cuda=False)
    _need(w, torch.float32, "w", 2, cuda=False)
    F, C = x.shape
    if F != dplan.n_fwd:
        raise ValueError("x has %d rows, the plan has %d forwarded positions" % (F, dplan.n_fwd))
    if w.shape[0] != C:
        raise ValueError("w must have shape (%d, W)" % C)
    y = torch.empty_like(x) if y is None else y
    _need(y, torch.bfloat16, "y", 2, cuda=False)
    _shape(y, (F, C), "y")
    _on_device(x, (w, "w"), (y, "y"), (dplan.image, "the plan image"))
    B.check(lib.tpk_gdn_conv(dplan.plan.handle, _ptr(dplan.image), _ptr(x), _ptr(w), _ptr(y), C, w.shape[1],
                             _stream()), "tpk_gdn_conv")
    return y


def gdn_delta_rule(dplan, q, k, v, g, beta, scale=None, out=None, workspace=None):
    """Gated delta rule along every root-to-leaf path (``tpk_gdn_delta_rule``).

    q, k [F, H, dk] and v [F, H, dv] bf16 -- views whose rows may be strided
    (e.g. column slices of the convolution's output), unit stride inside a
    row; g (log decay), beta [F, H] fp32.  Returns o [F, H, dv] bf16."""
    lib = B.load()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.dim() != 3:
            raise TypeError("%s must be a 3-d bf16 tensor" % n)
        if t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise ValueError("%s: heads and elements must be contiguous inside a row" % n)
    F, H, dk = q.shape
    dv = v.shape[2]
    if F != dplan.n_fwd:
        raise ValueError("q has %d rows, the plan has %d forwarded positions" % (F, dplan.n_fwd))
    _shape(k, (F, H, dk), "k")
    _shape(v, (F, H, dv), "v")
    if q.stride(0) != k.stride(0):
        raise ValueError("q and k must share one row stride")
    for t, n in ((g, "g"), (beta, "beta")):
        _need(t, torch.float32, n, 2, cuda=False)
        _shape(t, (F, H), n)
    scale = 1.0 / math.sqrt(dk) if scale is None else float(scale)
    out = torch.empty((F, H, dv), dtype=torch.bfloat16, device=q.device) if out is None else out
    _need(out, torch.bfloat16, "out", 3, cuda=False)
    _shape(out, (F, H, dv), "out")
    need = int(lib.tpk_gdn_workspace_bytes(dplan.plan.handle, H, dk, dv))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    if ws_bytes < need:
        raise ValueError("workspace has %d bytes, the delta rule needs %d" % (ws_bytes, need))
    _on_device(q, (k, "k"), (v, "v"), (g, "g"), (beta, "beta"), (out, "out"), (workspace, "workspace"),
               (dplan.image, "the plan image"))
    B.check(lib.tpk_gdn_delta_rule(dplan.plan.handle, _ptr(dplan.image), _ptr(q), _ptr(k), _ptr(v), q.stride(0),
                                   v.stride(0), _ptr(g), _ptr(beta), _ptr(out), H, dk, dv, scale, _ptr(workspace),
                                   ws_bytes, _stream()), "tpk_gdn_delta_rule")
    return out


def gdn_workspace(dplan, H, dk, dv):
    """A workspace for ``gdn_delta_rule`` (its saved per-instance final
    states); keep it for ``gdn_delta_rule_bwd``."""
    lib = B.load()
    need = int(lib.tpk_gdn_workspace_bytes(dplan.plan.handle, H, dk, dv))
    return torch.empty(max(need, 256), dtype=torch.uint8, device=dplan.image.device)


def _rows3(t, name, shape=None):
    """A 3-d bf16 view whose rows may be strided, contiguous inside a row."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.dim() != 3:
        raise TypeError("%s must be a 3-d bf16 tensor" % name)
    if shape is not None:
        _shape(t, shape, name)
    if t.stride(2) != 1 or t.stride(1) != t.shape[2]:
        raise ValueError("%s: heads and elements must be contiguous inside a row" % name)


def gdn_conv_bwd(dplan, x, w, dy, dx=None, dw=None, workspace=None):
    """Gradients of ``gdn_conv`` (``tpk_gdn_conv_bwd``): x, dy [F, C] bf16,
    w [C, W] fp32 -> (dx [F, C] bf16, dw [C, W] fp32)."""
    lib = B.load()
    _need(x, torch.bfloat16, "x", 2, cuda=False)
    _need(w, torch.float32, "w", 2, cuda=False)
    _need(dy, torch.bfloat16, "dy", 2, cuda=False)
    F, C = x.shape
    W = w.shape[1]
    if F != dplan.n_fwd:
        raise ValueError("x has %d rows, the plan has %d forwarded positions" % (F, dplan.n_fwd))
    if w.shape[0] != C:
        raise ValueError("w must have shape (%d, W)" % C)
    _shape(dy, (F, C), "dy")
    dx = torch.empty_like(x) if dx is None else dx
    dw = torch.empty_like(w) if dw is None else dw
    _need(dx, torch.bfloat16, "dx", 2, cuda=False)
    _shape(dx, (F, C), "dx")
    _need(dw, torch.float32, "dw", 2, cuda=False)
    _shape(dw, (C, W), "dw")
    need = int(lib.tpk_gdn_conv_bwd_workspace_bytes(dplan.plan.handle, C, W))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    if ws_bytes < need:
        raise ValueError("workspace has %d bytes, the convolution's backward needs %d" % (ws_bytes, need))
    _on_device(x, (w, "w"), (dy, "dy"), (dx, "dx"), (dw, "dw"), (workspace, "workspace"),
               (dplan.image, "the plan image"))
    B.check(lib.tpk_gdn_conv_bwd(dplan.plan.handle, _ptr(dplan.image), _ptr(x), _ptr(w), _ptr(dy), _ptr(dx), _ptr(dw),
                                 C, W, _ptr(workspace), ws_bytes, _stream()), "tpk_gdn_conv_bwd")
    return dx, dw


def gdn_delta_rule_bwd(dplan, q, k, v, g, beta, dout, state, scale=None, dq=None, dk=None, dv=None, dg=None,
                       dbeta=None, workspace=None):
    """Gradients of ``gdn_delta_rule`` (``tpk_gdn_delta_rule_bwd``).

    q, k, v, g, beta as given to the forward; ``state`` the workspace the
    forward filled; dout [F, H, dv] bf16.  dq, dk (sharing one row stride)
    and dv may be strided views, e.g. column slices of one [F, C] gradient.
    Returns (dq, dk, dv, dg, dbeta)."""
    lib = B.load()
    _rows3(q, "q")
    F, H, dkk = q.shape
    dvv = v.shape[2]
    if F != dplan.n_fwd:
        raise ValueError("q has %d rows, the plan has %d forwarded positions" % (F, dplan.n_fwd))
    _rows3(k, "k", (F, H, dkk))
    _rows3(v, "v", (F, H, dvv))
    if q.stride(0) != k.stride(0):
        raise ValueError("q and k must share one row stride")
    for t, n in ((g, "g"), (beta, "beta")):
        _need(t, torch.float32, n, 2, cuda=False)
        _shape(t, (F, H), n)
    _need(dout, torch.bfloat16, "dout", 3, cuda=False)
    _shape(dout, (F, H, dvv), "dout")
    dev = q.device
    dq = torch.empty((F, H, dkk), dtype=torch.bfloat16, device=dev) if dq is None else dq
    dk = torch.empty((F, H, dkk), dtype=torch.bfloat16, device=dev) if dk is None else dk
    dv = torch.empty((F, H, dvv), dtype=torch.bfloat16, device=dev) if dv is None else dv
    _rows3(dq, "dq", (F, H, dkk))
    _rows3(dk, "dk", (F, H, dkk))
    _rows3(dv, "dv", (F, H, dvv))
    if dq.stride(0) != dk.stride(0):
        raise ValueError("dq and dk must share one row stride")
    dg = torch.empty((F, H), dtype=torch.float32, device=dev) if dg is None else dg
    dbeta = torch.empty((F, H), dtype=torch.float32, device=dev) if dbeta is None else dbeta
    for t, n in ((dg, "dg"), (dbeta, "dbeta")):
        _need(t, torch.float32, n, 2, cuda=False)
        _shape(t, (F, H), n)
    if not isinstance(state, torch.Tensor):
        raise TypeError("state must be the forward's workspace tensor")
    st_bytes = state.numel() * state.element_size()
    need_st = int(lib.tpk_gdn_workspace_bytes(dplan.plan.handle, H, dkk, dvv))
    if st_bytes < need_st:
        raise ValueError("state has %d bytes, the forward's workspace has %d" % (st_bytes, need_st))
    need = int(lib.tpk_gdn_bwd_workspace_bytes(dplan.plan.handle, H, dkk, dvv))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size()
    if ws_bytes < need:
        raise ValueError("workspace has %d bytes, the delta rule's backward needs %d" % (ws_bytes, need))
    scale = 1.0 / math.sqrt(dkk) if scale is None else float(scale)
    _on_device(q, (k, "k"), (v, "v"), (g, "g"), (beta, "beta"), (dout, "dout"), (dq, "dq"), (dk, "dk"), (dv, "dv"),
               (dg, "dg"), (dbeta, "dbeta"), (state, "state"), (workspace, "workspace"),
               (dplan.image, "the plan image"))
    B.check(lib.tpk_gdn_delta_rule_bwd(dplan.plan.handle, _ptr(dplan.image), _ptr(q), _ptr(k), _ptr(v), q.stride(0),
                                       v.stride(0), _ptr(g), _ptr(beta), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                                       dq.stride(0), dv.stride(0), _ptr(dg), _ptr(dbeta), H, dkk, dvv, scale,
                                       _ptr(state), st_bytes, _ptr(workspace), ws_bytes, _stream()),
            "tpk_gdn_delta_rule_bwd")
    return dq, dk, dv, dg, dbeta


# ---- the operators around the token mixers ----------------------------------
#
# One token's call is a few microseconds of GPU work, so these wrappers check
# each tensor once (_arg) and hand plain addresses to ctypes.

_TABLE_TYPES = {torch.bfloat16: B.BF16, torch.float32: B.F32}


def _arg(t, dtype, shape, name):
    """t's address, once it is a contiguous tensor of dtype and shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _out(t, dtype, shape, name, ref):
    """(tensor, address) of an output: the caller's, checked, or a new one."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=ref.device)
        return t, t.data_ptr()
    return t, _arg(t, dtype, shape, name)


def _matrix(t, dtypes, name):
    """The shape of the 2-d tensor t, of one of dtypes, with rows of 8k channels."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype not in dtypes or t.dim() != 2:
        raise TypeError("%s must be a 2-d tensor of %s" % (name, " or ".join(str(d) for d in dtypes)))
    n, c = t.shape
    if c < 8 or c % 8:
        raise ValueError("%s must have a multiple of 8 channels, got %d" % (name, c))
    return n, c


def _device(names, *tensors):
    """The one CUDA device of the caller's tensors (None skipped).  Checked after
    the shapes, so a wrong shape is reported as such wherever the tensors live."""
    dev = tensors[0].get_device()
    for i, t in enumerate(tensors):
        if t is None:
            continue
        d = t.get_device()
        if d < 0:
            raise ValueError("%s must be a CUDA tensor (no CPU path exists)" % names.split()[i])
        if d != dev:
            raise ValueError("%s is on %s, expected cuda:%d" % (names.split()[i], t.device, dev))
    return dev


def _launch(dev, fn, *args):
    """fn(*args, stream) on device dev and that device's current stream."""
    if dev == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if st != B.TPK_OK:
        B.check(st, fn.__name__)


def _workspace(workspace, need, ref, what):
    """The caller's workspace tensor, checked, or a new one on ref's device."""
    if workspace is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=ref.device)
    if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor")
    if workspace.nbytes < need:
        raise ValueError("workspace has %d bytes, %s needs %d" % (workspace.nbytes, what, need))
    return workspace


def _dev_err(t):
    if t is None:
        return None
    _need(t, torch.int32, "dev_err", cuda=False)
    return t.data_ptr()


def embed(table, tokens, scale=1.0, out=None):
    """Embedding lookup with scaling (``tpk_embed``): out[f] = scale *
    table[tokens[f]] in bf16, a zero row where the id is outside the table.

    table [V, C] bf16 or fp32, tokens [N] int32 (e.g. ``gather_to_forwarded``
    of the raw token ids).  Returns out [N, C] bf16."""
    lib = B.load()
    V, C = _matrix(table, _TABLE_TYPES, "table")
    if V < 1:
        raise ValueError("table has no rows")
    p_table = _arg(table, table.dtype, (V, C), "table")
    N = tokens.numel() if isinstance(tokens, torch.Tensor) else 0
    p_tok = _arg(tokens, torch.int32, (N,), "tokens")
    given = out
    out, p_out = _out(out, torch.bfloat16, (N, C), "out", table)
    dev = _device("table tokens out", table, tokens, given)
    _launch(dev, lib.tpk_embed, p_table, _TABLE_TYPES[table.dtype], p_tok, p_out, N, V, C, float(scale))
    return out


def embed_bwd(tokens, dout, vocab, scale=1.0, dtype=torch.float32, dtable=None, workspace=None):
    """Gradient of ``embed``'s table (``tpk_embed_bwd``): dtable[v] = scale *
    sum of dout[f] over tokens[f] = v, fp32 sums in a fixed order; ids that do
    not occur get zero rows.

    tokens [N] int32, dout [N, C] bf16 -> dtable [vocab, C] of ``dtype`` (fp32
    or bf16; ignored if ``dtable`` is given)."""
    lib = B.load()
    N, C = _matrix(dout, (torch.bfloat16,), "dout")
    p_dout = _arg(dout, torch.bfloat16, (N, C), "dout")
    p_tok = _arg(tokens, torch.int32, (N,), "tokens")
    V = int(vocab)
    if V < 1:
        raise ValueError("vocab must be positive")
    dtype = dtype if dtable is None else dtable.dtype
    if dtype not in _TABLE_TYPES:
        raise TypeError("the table's gradient must be bf16 or fp32")
    given = dtable, workspace
    dtable, p_dt = _out(dtable, dtype, (V, C), "dtable", dout)
    ws = _workspace(workspace, lib.tpk_embed_bwd_workspace_bytes(N, V, C), dout, "the lookup's backward")
    dev = _device("dout tokens dtable workspace", dout, tokens, *given)
    _launch(dev, lib.tpk_embed_bwd, p_tok, p_dout, p_dt, _TABLE_TYPES[dtype], N, V, C, float(scale), ws.data_ptr(),
            ws.nbytes)
    return dtable


def _onto(p_res, ld_res, p_out, ld_out):
    """``out`` may be the residual, row for row."""
    if p_res == p_out and p_res is not None and ld_res != ld_out:
        raise ValueError("out starts where residual does, with other rows")


def _row_stride(ld, rows, width, name):
    """The stride of rows of ``width`` elements that may lie apart (column slices),
    given as ld elements: 16-byte aligned, without overlap; of no account for one row."""
    if rows <= 1:
        return width
    if ld < width or ld % 8:
        raise ValueError("%s: rows must not overlap and must lie a multiple of 8 elements apart" % name)
    return ld


def _rows2(t, name, shape):
    """(address, row stride in elements) of a 2-d bf16 tensor whose rows may
    lie apart (column slices), 16-byte aligned."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.dim() != 2:
        raise TypeError("%s must be a 2-d bf16 tensor" % name)
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    ld, unit = t.stride()
    if unit != 1:
        raise ValueError("%s: channels must be contiguous inside a row" % name)
    return t.data_ptr(), _row_stride(ld, shape[0], shape[1], name)


def _norm_args(res, w_pre, y, w_post, gate):
    """(shape, the inputs' addresses and row strides in the C call's order)."""
    shape = _matrix(res, (torch.bfloat16,), "res")
    C = shape[1]
    p_res = _arg(res, torch.bfloat16, shape, "res")
    if y is None:
        if gate is not None or w_post is not None:
            raise ValueError("gate and w_post apply to y, which is missing")
        p_y, ld_y = None, C
    else:
        p_y, ld_y = _rows2(y, "y", shape)
    p_gate, ld_gate = (None, C) if gate is None else _rows2(gate, "gate", shape)
    p_post = None if w_post is None else _arg(w_post, torch.float32, (C,), "w_post")
    return shape, (p_res, p_y, ld_y, p_gate, ld_gate, p_post, _arg(w_pre, torch.float32, (C,), "w_pre"))


def block_norm(res, w_pre, y=None, w_post=None, gate=None, scale=1.0, eps=1e-6, res_out=None, out=None):
    """The norms around a block with its gate and residual (``tpk_block_norm``):

        r = res + scale * sigmoid(gate) * rmsnorm(y) * w_post
        x = rmsnorm(r) * w_pre

    res [N, C] bf16 (residual stream), y [N, C] bf16 (the block's output) and
    gate [N, C] bf16, whose rows may be strided (column slices); w_pre, w_post
    [C] fp32.  Without w_post y enters as it is, without gate the sigmoid is
    1; without y (the norm before the first block) r is res.  Returns
    (r, x), both [N, C] bf16; ``res_out`` may be ``res`` itself."""
    lib = B.load()
    shape, args = _norm_args(res, w_pre, y, w_post, gate)
    if y is None and res_out is not None:
        raise ValueError("without y nothing is added to res: res_out is not written")
    given = res_out, out
    res_out, p_ro = (None, None) if y is None else _out(res_out, torch.bfloat16, shape, "res_out", res)
    out, p_out = _out(out, torch.bfloat16, shape, "out", res)
    dev = _device("res w_pre y w_post gate res_out out", res, w_pre, y, w_post, gate, *given)
    _launch(dev, lib.tpk_block_norm, *args, p_ro, p_out, *shape, float(scale), float(eps))
    return (res if y is None else res_out), out


def block_norm_bwd(res, w_pre, dx, dres_out=None, y=None, w_post=None, gate=None, scale=1.0, eps=1e-6, dres=None,
                   dy=None, dgate=None, dw_post=None, dw_pre=None, workspace=None):
    """Gradients of ``block_norm`` (``tpk_block_norm_bwd``) for the gradients
    dx of x and dres_out of r (None: none); the other inputs as given to the
    forward.  dy and dgate may be column slices of a wider gradient.  Returns
    (dres, dy, dgate, dw_post, dw_pre), None where the input was None."""
    lib = B.load()
    shape, args = _norm_args(res, w_pre, y, w_post, gate)
    C = shape[1]
    p_dx = _arg(dx, torch.bfloat16, shape, "dx")
    p_dro = None if dres_out is None else _arg(dres_out, torch.bfloat16, shape, "dres_out")
    for t, n, ref in ((dy, "dy", y), (dgate, "dgate", gate), (dw_post, "dw_post", w_post)):
        if t is not None and ref is None:
            raise ValueError("%s is given, but not the input it is the gradient of" % n)
    given = dres, dy, dgate, dw_post, dw_pre, workspace
    bf16 = torch.bfloat16
    dres, p_dres = _out(dres, bf16, shape, "dres", res)
    p_dy = p_dgate = p_dpost = None
    ld_dy = ld_dgate = C
    if dy is not None:
        p_dy, ld_dy = _rows2(dy, "dy", shape)
    elif y is not None:
        dy, p_dy = _out(None, bf16, shape, "dy", res)
    if dgate is not None:
        p_dgate, ld_dgate = _rows2(dgate, "dgate", shape)
    elif gate is not None:
        dgate, p_dgate = _out(None, bf16, shape, "dgate", res)
    if w_post is not None:
        dw_post, p_dpost = _out(dw_post, torch.float32, (C,), "dw_post", res)
    dw_pre, p_dpre = _out(dw_pre, torch.float32, (C,), "dw_pre", res)
    ws = _workspace(workspace, lib.tpk_block_norm_bwd_workspace_bytes(*shape), res, "the norms' backward")
    dev = _device("res w_pre dx dres_out y w_post gate dres dy dgate dw_post dw_pre workspace", res, w_pre, dx,
                  dres_out, y, w_post, gate, *given)
    _launch(dev, lib.tpk_block_norm_bwd, *args, p_dro, p_dx, p_dres, p_dy, ld_dy, p_dgate, ld_dgate, p_dpost, p_dpre,
            *shape, float(scale), float(eps), ws.data_ptr(), ws.nbytes)
    return dres, dy, dgate, dw_post, dw_pre


def _loss_args(h, w, target, scale):
    """(N, V, C, addresses of h, w, target), checked."""
    N, C = _matrix(h, (torch.bfloat16,), "h")
    V = _matrix(w, (torch.bfloat16,), "w")[0]
    if V < 1:
        raise ValueError("w has no rows")
    if not 0.0 < scale < math.inf:
        raise ValueError("scale must be positive and finite")
    return N, V, C, (_arg(h, torch.bfloat16, (N, C), "h"), _arg(w, torch.bfloat16, (V, C), "w"),
                     _arg(target, torch.int32, (N,), "target"))


def lm_loss(h, w, target, scale=1.0, loss=None, lse=None, workspace=None, dev_err=None):
    """Softmax cross entropy over the vocabulary without the logits (``tpk_lm_loss``).

    h [N, C] bf16 (hidden rows), w [V, C] bf16 (output projection), target [N]
    int32; logits are ``scale * h @ w.T`` (scale = 1 / temperature).  Returns
    (loss, lse), fp32 [N]: loss = lse - logit[target], both zero where the
    target is outside [0, V) (a position without a prediction).  A device wait
    that gives up is reported in ``dev_err`` (int32) alone."""
    lib = B.load()
    N, V, C, args = _loss_args(h, w, target, scale)
    given = loss, lse, workspace, dev_err
    loss, p_loss = _out(loss, torch.float32, (N,), "loss", h)
    lse, p_lse = _out(lse, torch.float32, (N,), "lse", h)
    p_err = _dev_err(dev_err)
    ws = _workspace(workspace, lib.tpk_lm_loss_workspace_bytes(N, V, C, 0), h, "the loss")
    dev = _device("h w target loss lse workspace dev_err", h, w, target, *given)
    _launch(dev, lib.tpk_lm_loss, *args, p_loss, p_lse, N, V, C, float(scale), ws.data_ptr(), ws.nbytes, p_err)
    return loss, lse


def lm_loss_bwd(h, w, target, lse, dloss, scale=1.0, dh=None, dw=None, workspace=None, dev_err=None):
    """Gradients of sum(dloss * loss) (``tpk_lm_loss_bwd``): h, w, target,
    scale as given to ``lm_loss``, lse its result for these rows in one call (it
    has to fit the scores, which are computed again), dloss [N] fp32 the weight
    of each position's loss (e.g. ``sum_to_forwarded`` of per-token weights).
    Returns (dh [N, C] bf16, dw [V, C] bf16)."""
    lib = B.load()
    N, V, C, args = _loss_args(h, w, target, scale)
    p_lse, p_dloss = _arg(lse, torch.float32, (N,), "lse"), _arg(dloss, torch.float32, (N,), "dloss")
    given = dh, dw, workspace, dev_err
    dh, p_dh = _out(dh, torch.bfloat16, (N, C), "dh", h)
    dw, p_dw = _out(dw, torch.bfloat16, (V, C), "dw", h)
    p_err = _dev_err(dev_err)
    ws = _workspace(workspace, lib.tpk_lm_loss_workspace_bytes(N, V, C, 1), h, "the loss's backward")
    dev = _device("h w target lse dloss dh dw workspace dev_err", h, w, target, lse, dloss, *given)
    _launch(dev, lib.tpk_lm_loss_bwd, *args, p_lse, p_dloss, p_dh, p_dw, N, V, C, float(scale), ws.data_ptr(),
            ws.nbytes, p_err)
    return dh, dw


# ---- projections, feed-forward block, rotary positions, policy objective --------

ACTIVATIONS = {"none": B.ACT_NONE, None: B.ACT_NONE, "silu": B.ACT_SILU, "gelu": B.ACT_GELU,
               "gelu_tanh": B.ACT_GELU_TANH}


def _activation(name):
    if name not in ACTIVATIONS:
        raise ValueError("act must be one of none, silu, gelu, gelu_tanh, got %r" % (name,))
    return ACTIVATIONS[name]


def _out_rows(t, shape, name, ref):
    """(tensor, address, row stride) of a bf16 output whose rows may lie apart."""
    if t is None:
        t = torch.empty(shape, dtype=torch.bfloat16, device=ref.device)
        return t, t.data_ptr(), shape[1]
    return (t,) + _rows2(t, name, shape)


def _rows_of(t, name):
    """(rows, channels, address, row stride) of a 2-d bf16 tensor whose rows may
    lie apart, of a multiple of 8 channels."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.dim() != 2:
        raise TypeError("%s must be a 2-d bf16 tensor" % name)
    n, c = t.shape
    if c < 8 or c % 8:
        raise ValueError("%s must have a multiple of 8 channels, got %d" % (name, c))
    ld, unit = t.stride()
    if unit != 1:
        raise ValueError("%s: channels must be contiguous inside a row" % name)
    return n, c, t.data_ptr(), _row_stride(ld, n, c, name)


def _weights(t, cols, name):
    """(rows, address) of a contiguous bf16 matrix of `cols` columns and a multiple of 8 rows."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.dim() != 2:
        raise TypeError("%s must be a 2-d bf16 tensor" % name)
    rows, c = t.shape
    if c != cols:
        raise ValueError("%s must have shape (rows, %d), got %s" % (name, cols, tuple(t.shape)))
    if rows < 8 or rows % 8:
        raise ValueError("%s must have a multiple of 8 rows, got %d" % (name, rows))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return rows, t.data_ptr()


def _linear_args(x, w, bias):
    """(N, C, O, addresses and stride of x, w, bias), checked."""
    N, C, p_x, ld_x = _rows_of(x, "x")
    O, p_w = _weights(w, C, "w")
    return N, C, O, p_x, ld_x, p_w, None if bias is None else _arg(bias, torch.float32, (O,), "bias")


def linear(x, w, bias=None, act="none", residual=None, out=None, workspace=None, dev_err=None):
    """Matrix product with bias, activation and residual (``tpk_linear``):
    y = act(x @ w.T + bias) + residual.

    x [N, C], w [O, C], residual [N, O] bf16, bias [O] fp32; rows of x, residual
    and ``out`` may be strided (column slices).  act: none, silu, gelu or
    gelu_tanh.  ``out`` may be ``residual``.  Returns y [N, O] bf16."""
    lib = B.load()
    N, C, O, p_x, ld_x, p_w, p_b = _linear_args(x, w, bias)
    a = _activation(act)
    p_r, ld_r = (None, O) if residual is None else _rows2(residual, "residual", (N, O))
    given = out, workspace, dev_err
    out, p_y, ld_y = _out_rows(out, (N, O), "out", x)
    _onto(p_r, ld_r, p_y, ld_y)
    p_err = _dev_err(dev_err)
    # (a few rows, one or so, are a matter of microseconds: no question about a workspace they do not need)
    need = 0 if N <= B.FEW_ROWS else lib.tpk_linear_workspace_bytes(N, C, O, a, 0)
    ws = _workspace(workspace, need, x, "the projection") if need or workspace is not None else None
    dev = _device("x w bias residual out workspace dev_err", x, w, bias, residual, *given)
    _launch(dev, lib.tpk_linear, p_x, ld_x, p_w, p_b, a, p_r, ld_r, p_y, ld_y, N, C, O,
            None if ws is None else ws.data_ptr(), 0 if ws is None else ws.nbytes, p_err)
    return out


def linear_bwd(x, w, dy, bias=None, act="none", dx=None, dw=None, db=None, workspace=None, dev_err=None):
    """Gradients of ``linear`` for the gradient dy of its result
    (``tpk_linear_bwd``); x, w, bias, act as given to it.  The residual's
    gradient is dy.  With an activation x @ w.T + bias is formed again.  dy and
    ``dx`` may be column slices.  Returns (dx [N, C] bf16, dw [O, C] bf16,
    db [O] fp32, None without a bias)."""
    lib = B.load()
    N, C, O, p_x, ld_x, p_w, p_b = _linear_args(x, w, bias)
    a = _activation(act)
    p_dy, ld_dy = _rows2(dy, "dy", (N, O))
    if db is not None and bias is None:
        raise ValueError("db is given, but not the bias it is the gradient of")
    given = dx, dw, db, workspace, dev_err
    dx, p_dx, ld_dx = _out_rows(dx, (N, C), "dx", x)
    dw, p_dw = _out(dw, torch.bfloat16, (O, C), "dw", x)
    db, p_db = (None, None) if bias is None else _out(db, torch.float32, (O,), "db", x)
    p_err = _dev_err(dev_err)
    ws = _workspace(workspace, lib.tpk_linear_workspace_bytes(N, C, O, a, 1), x, "the projection's backward")
    dev = _device("x w dy bias dx dw db workspace dev_err", x, w, dy, bias, *given)
    _launch(dev, lib.tpk_linear_bwd, p_x, ld_x, p_w, p_b, a, p_dy, ld_dy, p_dx, ld_dx, p_dw, p_db, N, C, O,
            ws.data_ptr(), ws.nbytes, p_err)
    return dx, dw, db


def linear_plan(n, c, o, act="none", backward=False):
    """How ``linear`` (or ``linear_bwd``) does the products of n rows, c channels
    and o results (``tpk_linear_plan``): {"y" / "dz", "dx", "dw": {"form": few,
    wide, narrow or together, "teams", "tiles", "split_tiles", "splits",
    "pieces"}}.  For profiles and tests; needs no GPU."""
    out = (B.ProductPlan * 3)()
    got = B.load().tpk_linear_plan(n, c, o, _activation(act), 1 if backward else 0, out)
    if got < 0:
        B.check(got, "tpk_linear_plan")
    plans = {}
    for p in out[:got]:
        d = {k: getattr(p, k) for k, _ in p._fields_[2:]}
        plans[B.PRODUCTS[p.product]] = dict(form=B.FORMS[p.form], **d)
    return plans


def _ffn_args(x, w_in, w_out):
    """(N, C, I, O, address and stride of x, addresses of the weights), checked."""
    N, C, p_x, ld_x = _rows_of(x, "x")
    I2, p_in = _weights(w_in, C, "w_in")
    if I2 % 16:
        raise ValueError("w_in must have twice a multiple of 8 rows, got %d" % I2)
    O, p_out = _weights(w_out, I2 // 2, "w_out")
    return N, C, I2 // 2, O, p_x, ld_x, p_in, p_out


def gated_ffn(x, w_in, w_out, act="silu", residual=None, save=False, out=None, pre=None, a=None, workspace=None,
              dev_err=None):
    """Gated feed-forward block (``tpk_gated_ffn``):
    y = (act(x @ w_in[:I].T) * (x @ w_in[I:].T)) @ w_out.T + residual.

    x [N, C], w_in [2 I, C] (the gate's rows first), w_out [O, I], residual
    [N, O] bf16; rows of x, residual and ``out`` may be strided; ``out`` may be
    ``residual``.  Returns y [N, O]; with ``save`` (y, pre, a), what
    ``gated_ffn_bwd`` needs: pre uint8, g and u in a form of the library's own,
    a [N, I] bf16."""
    lib = B.load()
    N, C, I, O, p_x, ld_x, p_in, p_out = _ffn_args(x, w_in, w_out)
    k = _activation(act)
    if not save and (pre is not None or a is not None):
        raise ValueError("pre and a are written with save=True alone")
    p_r, ld_r = (None, O) if residual is None else _rows2(residual, "residual", (N, O))
    given = out, pre, a, workspace, dev_err
    out, p_y, ld_y = _out_rows(out, (N, O), "out", x)
    _onto(p_r, ld_r, p_y, ld_y)
    p_pre = p_a = None
    if save:
        pre, p_pre = _out(pre, torch.uint8, (lib.tpk_gated_ffn_saved_bytes(N, I),), "pre", x)
        a, p_a = _out(a, torch.bfloat16, (N, I), "a", x)
    p_err = _dev_err(dev_err)
    ws = _workspace(workspace, lib.tpk_gated_ffn_workspace_bytes(N, C, I, O, 0), x, "the block")
    dev = _device("x w_in w_out residual out pre a workspace dev_err", x, w_in, w_out, residual, *given)
    _launch(dev, lib.tpk_gated_ffn, p_x, ld_x, p_in, p_out, k, p_r, ld_r, p_pre, p_a, p_y, ld_y, N, C, I, O,
            ws.data_ptr(), ws.nbytes, p_err)
    return (out, pre, a) if save else out


def gated_ffn_bwd(x, w_in, w_out, dy, pre, a, act="silu", dx=None, dw_in=None, dw_out=None, workspace=None,
                  dev_err=None):
    """Gradients of ``gated_ffn`` for the gradient dy of its result
    (``tpk_gated_ffn_bwd``); x, the weights and act as given to it, pre and a
    as it saved them.  The residual's gradient is dy.  dy and ``dx`` may be
    column slices.  Returns (dx [N, C], dw_in [2 I, C], dw_out [O, I]) bf16."""
    lib = B.load()
    N, C, I, O, p_x, ld_x, p_in, p_out = _ffn_args(x, w_in, w_out)
    k = _activation(act)
    p_dy, ld_dy = _rows2(dy, "dy", (N, O))
    p_pre = _arg(pre, torch.uint8, (lib.tpk_gated_ffn_saved_bytes(N, I),), "pre")
    p_a = _arg(a, torch.bfloat16, (N, I), "a")
    given = dx, dw_in, dw_out, workspace, dev_err
    dx, p_dx, ld_dx = _out_rows(dx, (N, C), "dx", x)
    dw_in, p_din = _out(dw_in, torch.bfloat16, (2 * I, C), "dw_in", x)
    dw_out, p_dout = _out(dw_out, torch.bfloat16, (O, I), "dw_out", x)
    p_err = _dev_err(dev_err)
    ws = _workspace(workspace, lib.tpk_gated_ffn_workspace_bytes(N, C, I, O, 1), x, "the block's backward")
    dev = _device("x w_in w_out dy pre a dx dw_in dw_out workspace dev_err", x, w_in, w_out, dy, pre, a, *given)
    _launch(dev, lib.tpk_gated_ffn_bwd, p_x, ld_x, p_in, p_out, k, p_dy, ld_dy, p_pre, p_a, p_dx, ld_dx, p_din, p_dout,
            N, C, I, O, ws.data_ptr(), ws.nbytes, p_err)
    return dx, dw_in, dw_out


def rope_freqs(rot, base=1e4, stretch=1.0, trained=None, fast=32.0, slow=1.0):
    """Radians per position of each of the rot / 2 pairs (float64), for
    ``rope_by_depth_ex``: base^(-2i / rot), stretched for contexts ``stretch``
    times as long as the model was trained on.  Without ``trained`` every
    frequency is divided by stretch (positions interpolated); with ``trained``
    (that context's length) pairs that turn ``fast`` times or more in it keep
    theirs, those that turn ``slow`` times or less are divided, with a linear
    ramp between."""
    f = float(base) ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if trained is None:
        return f / stretch
    if not fast > slow:
        raise ValueError("fast must be above slow")
    keep = np.clip((trained * f / (2.0 * np.pi) - slow) / (fast - slow), 0.0, 1.0)
    return f * (keep + (1.0 - keep) / stretch)


def _heads(t, name):
    """(positions, heads, channels, address, row stride) of a 3-d bf16 tensor whose rows may lie apart."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.dim() != 3:
        raise TypeError("%s must be a 3-d bf16 tensor" % name)
    n, h, d = t.shape
    ld, head, unit = t.stride()
    if unit != 1 or head != d:
        raise ValueError("%s: heads and elements must be contiguous inside a row" % name)
    return n, h, d, t.data_ptr(), _row_stride(ld, n, h * d, name)


def _rotated(t, out, name, F, d):
    """(heads, address, row stride, output, its address, its row stride) of q or k and what it turns into."""
    if t is None:
        if out is not None:
            raise ValueError("%s_out is given, but not %s" % (name, name))
        return 0, None, 0, None, None, 0
    n, h, c, p_in, ld_in = _heads(t, name)
    if n != F or c != d:
        raise ValueError("%s must have shape %s, got %s" % (name, (F, h, d), (n, h, c)))
    if out is None:
        out = torch.empty((n, h, c), dtype=torch.bfloat16, device=t.device)
        return h, p_in, ld_in, out, out.data_ptr(), h * c
    n, ho, c, p_out, ld_out = _heads(out, name + "_out")
    if n != F or ho != h or c != d:
        raise ValueError("%s_out must have shape %s, got %s" % (name, (F, h, d), (n, ho, c)))
    if p_out == p_in and ld_out != ld_in:
        raise ValueError("%s_out starts where %s does, with other rows" % (name, name))
    return h, p_in, ld_in, out, p_out, ld_out


def rope_by_depth_ex(q, k, depth, freqs, interleaved=False, factor=1.0, inverse=False, q_out=None, k_out=None):
    """RoPE at ``depth`` in its other forms (``tpk_rope_by_depth_ex``): either
    pairing of channels (halves, or ``interleaved`` neighbours), in the first
    ``2 * len(freqs)`` channels of a head, by ``depth * freqs`` radians
    (``rope_freqs``), times ``factor``; the other channels are copied.
    ``inverse``: the transpose, for gradients.

    q [F, Hq, d], k [F, Hkv, d] bf16 (either may be None), rows may be strided
    (column slices of a fused projection); depth int32 [F].  Returns
    (q_out, k_out), new contiguous tensors unless given; ``q_out=q`` rotates in
    place."""
    lib = B.load()
    if q is None and k is None:
        return None, None
    ref = q if q is not None else k
    if not isinstance(ref, torch.Tensor) or ref.dim() != 3:
        raise TypeError("q and k must be 3-d bf16 tensors")
    F, _, d = ref.shape
    fr = np.ascontiguousarray(freqs, dtype=np.float64)
    pairs = len(fr) if fr.ndim == 1 else 0
    if pairs % 8 or not 8 <= pairs <= 128 or 2 * pairs > d:
        raise ValueError("freqs must hold a multiple of 8 pairs, no more than half the head (or 128)")
    if d % 8 or d > 512:
        raise ValueError("heads must have a multiple of 8 channels, 512 at most, got %d" % d)
    p_depth = _arg(depth, torch.int32, (F,), "depth")
    hq, p_q, ld_q, q_new, p_qo, ld_qo = _rotated(q, q_out, "q", F, d)
    hk, p_k, ld_k, k_new, p_ko, ld_ko = _rotated(k, k_out, "k", F, d)
    dev = _device("depth q k q_out k_out", depth, q, k, q_out, k_out)
    opts = B.RopeOpts(2 * pairs, 1 if interleaved else 0, float(factor), fr.__array_interface__["data"][0])
    _launch(dev, lib.tpk_rope_by_depth_ex, p_q, ld_q, p_k, ld_k, p_qo, ld_qo, p_ko, ld_ko, p_depth, F, hq, hk, d,
            ctypes.byref(opts), 1 if inverse else 0)
    return q_new, k_new


def policy_loss(loss, old_logp, advantage, weight, token_index, fwd_raw_begin, fwd_raw, ref_logp=None, clip_low=0.2,
                clip_high=0.2, dual_clip=0.0, kl_coef=0.0, seq_offsets=None, stats=None, dloss=None, workspace=None):
    """Clipped policy objective with a KL term over a packed batch, and its
    gradient with respect to ``lm_loss``'s loss (``tpk_policy_loss``).

    loss [F] fp32 (``lm_loss``: minus the log-probabilities); per raw token
    old_logp, advantage, weight and optionally ref_logp [R] fp32 (a weight of 0:
    no loss, nothing else of the token is read); token_index, fwd_raw_begin,
    fwd_raw: a device plan's.  The ratio is a token's, or with ``seq_offsets``
    (int32 [sequences + 1]) the geometric mean over its sequence.  clip_low,
    clip_high: the ratio's band around 1; dual_clip > 1: the ratio's limit where
    the advantage is negative; kl_coef: weight of exp(t) - t - 1, t = ref - logp.
    Returns (stats, dloss): stats [5] fp32 = the objective, weighted sums of the
    KL term, of the clipped tokens and of the ratio, the sum of weights; dloss
    [F] fp32, for ``lm_loss_bwd``."""
    lib = B.load()
    f32, i32 = torch.float32, torch.int32
    if not isinstance(loss, torch.Tensor) or not isinstance(old_logp, torch.Tensor):
        raise TypeError("loss and old_logp must be tensors")
    F, R = loss.numel(), old_logp.numel()
    args = (_arg(loss, f32, (F,), "loss"), _arg(old_logp, f32, (R,), "old_logp"),
            None if ref_logp is None else _arg(ref_logp, f32, (R,), "ref_logp"),
            _arg(advantage, f32, (R,), "advantage"), _arg(weight, f32, (R,), "weight"),
            _arg(token_index, i32, (R,), "token_index"), _arg(fwd_raw_begin, i32, (F + 1,), "fwd_raw_begin"),
            _arg(fwd_raw, i32, (R,), "fwd_raw"))
    if F > R:
        raise ValueError("loss has %d positions, more than the %d raw tokens" % (F, R))
    if not 0.0 <= clip_low <= 1.0 or not clip_high >= 0.0 or not (dual_clip == 0.0 or dual_clip > 1.0) or \
            not 0.0 <= kl_coef < math.inf:
        raise ValueError("clip_low must be in [0, 1], clip_high >= 0, dual_clip 0 or above 1, kl_coef >= 0")
    seqs, p_seq = 0, None
    if seq_offsets is not None:
        seqs = seq_offsets.numel() - 1 if isinstance(seq_offsets, torch.Tensor) else 0
        p_seq = _arg(seq_offsets, i32, (seqs + 1,), "seq_offsets")
        if seqs < 1:
            raise ValueError("seq_offsets must hold at least one sequence")
    given = stats, dloss, workspace
    stats, p_stats = _out(stats, f32, (5,), "stats", loss)
    dloss, p_dloss = _out(dloss, f32, (F,), "dloss", loss)
    ws = _workspace(workspace, lib.tpk_policy_loss_workspace_bytes(R, seqs), loss, "the objective")
    dev = _device("loss old_logp advantage weight token_index fwd_raw_begin fwd_raw ref_logp seq_offsets stats dloss "
                  "workspace", loss, old_logp, advantage, weight, token_index, fwd_raw_begin, fwd_raw, ref_logp,
                  seq_offsets, *given)
    opts = B.PolicyOpts(float(clip_low), float(clip_high), float(dual_clip), float(kl_coef))
    _launch(dev, lib.tpk_policy_loss, *args, p_seq, seqs, ctypes.byref(opts), p_stats, p_dloss, R, F, ws.data_ptr(),
            ws.nbytes)
    return stats, dloss
