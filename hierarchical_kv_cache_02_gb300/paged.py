"""A KV cache in pages of the caller's device memory, and the operators of a speculative decoding step on it.

    rope = RopeTable(128, theta=10000.0)
    kv = PagedKV(cfg, pages, table)
    q = kv.append(k, v, cu, lens, rope, rope_pos=lens_of_tokens + depth, q=q)  # the drafts' records at [len, len + T)
    out = kv.tree_attn(q.view(R, T, Hq, D), lens, tree_mask(parents))     # all nodes at once
    kv.keep_path(lens, path, count)                                       # the accepted ones move up
    lens += count

Every method only checks and marshals its arguments and calls the matching hs_* entry point; the work runs
in the library's kernels on the given (or current) stream, without allocating device memory beyond the
outputs and the workspace of a call, and can be captured in a CUDA graph.
"""
from __future__ import annotations

import ctypes

from . import _lib
from .pool import HsConfig, HsError, _check, _dev_tensor, _fast_ptr, _fast_stream, _tree_args


class RopeTable:
    """Frequencies of a rotary embedding on one device, as fractions of a turn per position.

    rotary_dim: rotated values of a head, a multiple of 16.  inv_freq: rotary_dim / 2 angles per position
    (radians); default theta ** (-2 j / rotary_dim).  interleaved: value 2j turns with 2j + 1, else j with
    j + rotary_dim / 2.  axes: for positions with several axes (time, row and column of an image, say), the axis of each
    of the rotary_dim / 2 pairs, numbers from 0 on, at most 4 of them; tokens then have a position for each axis."""

    def __init__(self, rotary_dim: int, theta: float = 10000.0, inv_freq=None, interleaved: bool = False,
                 device: int = 0, axes=None):
        import numpy as np
        import torch

        if rotary_dim < 16 or rotary_dim % 16 != 0:
            raise ValueError("rotary_dim must be a positive multiple of 16")
        half = rotary_dim // 2
        if inv_freq is None:
            inv_freq = [float(theta) ** (-j / half) for j in range(half)]
        f = np.ascontiguousarray(inv_freq, dtype=np.float64)
        if f.shape != (half,):
            raise ValueError(f"inv_freq must hold {half} values")
        turns = np.empty((half,), dtype=np.uint64)
        _check("hs_rope_turns", _lib.load().hs_rope_turns(f.ctypes.data, half, turns.ctypes.data))
        self.rotary_dim, self.interleaved, self.device = int(rotary_dim), bool(interleaved), int(device)
        self.axes, self.axis = 1, None
        if axes is not None:
            a = np.asarray(axes)
            if a.shape != (half,) or a.dtype.kind not in "iu" or a.min() < 0 or a.max() >= _lib.MAX_AXES:
                raise ValueError(f"axes must hold {half} numbers from 0 to {_lib.MAX_AXES - 1}")
            self.axes = int(a.max()) + 1
        self.turns = torch.from_numpy(turns.view(np.int64)).to(f"cuda:{self.device}")
        if self.axes > 1:
            self.axis = torch.from_numpy(a.astype(np.uint8)).to(f"cuda:{self.device}")


def tree_mask(parents):
    """Visibility of a tree: parents int [R][T] (-1: a child of the last context token) -> int64
    [R][T][ceil(T/64)], bit j of node i's words set when j is i or an ancestor of i."""
    import torch

    if parents.dim() != 2:
        raise ValueError("parents must be [R][T]")
    R, T = parents.shape
    j = torch.arange(T, device=parents.device)
    sees = (parents[:, :, None] == j) | (j[:, None] == j)
    reach = 1
    while reach < T:  # the square of a reachability matrix reaches twice as far
        sees = torch.bmm(sees.float(), sees.float()) > 0
        reach *= 2
    words = (T + 63) // 64
    bits = torch.zeros((R, T, words * 64), dtype=torch.int64, device=parents.device)
    bits[:, :, :T] = sees
    return (bits.view(R, T, words, 64) << torch.arange(64, device=parents.device)).sum(dim=3)


def _strided(torch, t, n, heads, dim, name, device, written=False):
    """Pointer, token stride and head stride of a bf16 [n][heads][dim] view ([n][dim] when heads is 1)."""
    try:
        if t.dtype is torch.bfloat16 and t.shape == (n, heads, dim) and t.get_device() == device:
            ts, hs, vs = t.stride()
            p = t.data_ptr()
            if vs == 1 and n > 1 and heads > 1 and not (ts | hs | p >> 1) & 7 and (not written or ts >= (heads - 1) * hs + dim):
                return p, ts, hs  # what most calls pass; the rest is looked at one by one
    except AttributeError:
        pass

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda" or t.device.index != device:
        raise ValueError(f"{name} must live on cuda:{device}")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    shape, st = tuple(t.shape), t.stride()
    if shape == (n, dim) and heads == 1:
        shape, st = (n, 1, dim), (st[0], 0, st[1])
    if shape != (n, heads, dim):
        raise ValueError(f"{name} must have shape {(n, heads, dim)}, got {tuple(t.shape)}")
    if st[2] != 1:
        raise ValueError(f"the values of a head of {name} must be contiguous")
    ts, hs = st[0] if n > 1 else 0, st[1] if heads > 1 else 0
    if ts % 8 or hs % 8 or t.data_ptr() % 16:
        raise ValueError(f"{name}: address and strides must be multiples of 16 bytes")
    if written and ((n > 1 and ts < dim) or (heads > 1 and hs < dim) or
                    (n > 1 and heads > 1 and ts < (heads - 1) * hs + dim and hs < (n - 1) * ts + dim)):
        raise ValueError(f"{name} must not overlap itself")
    return t.data_ptr(), ts, hs


def _weights(torch, t, heads, dim, name, device):
    """Pointer, head stride and type of a norm's weights [dim] or [heads][dim], bf16 or float32."""
    if t is None:
        return 0, 0, 0
    if not isinstance(t, torch.Tensor) or (t.dtype is not torch.bfloat16 and t.dtype is not torch.float32):
        raise TypeError(f"{name} must be a torch.Tensor of bfloat16 or float32")
    several = t.dim() == 2
    p = _fast_ptr(t, t.dtype, (heads, dim) if several else (dim,), name, device)
    if p & 15:
        raise ValueError(f"{name} must be aligned to 16 bytes")
    return p, dim if several else 0, _lib.WEIGHT_FP32 if t.dtype is torch.float32 else _lib.WEIGHT_BF16


class PagedKV:
    """pages bf16 [num_pages][page_tokens][record_elems] on a GPU; table int32 [R][max_pages]: position p
    of request r is row p % page_tokens of page table[r][p // page_tokens]; without a table request r owns
    the pages [r * max_pages, (r + 1) * max_pages).  Of cfg only num_requests (R), layout and the head
    counts and sizes are read.  Both tensors stay the caller's, who may change them between calls."""

    def __init__(self, cfg: HsConfig, pages, table=None):
        import torch

        if not isinstance(pages, torch.Tensor) or pages.device.type != "cuda" or pages.dim() != 3:
            raise ValueError("pages must be a CUDA tensor [num_pages][page_tokens][record_elems]")
        self.lib = _lib.load()
        self.cfg, self.device = cfg, pages.device.index
        self._c = cfg.to_c()
        self._tree_sizes = {}
        R = cfg.num_requests
        p = _dev_tensor(pages, torch.bfloat16, (pages.shape[0], pages.shape[1], cfg.record_elems), "pages", self.device)
        t = None
        if table is not None:
            if table.dim() != 2:
                raise ValueError("table must be [R][max_pages]")
            t = _dev_tensor(table, torch.int32, (R, table.shape[1]), "table", self.device)
            max_pages = int(table.shape[1])
        else:
            if pages.shape[0] % R:
                raise ValueError("without a table the pages must divide evenly among the requests")
            max_pages = pages.shape[0] // R
        self.pages, self.table = pages, table
        self._err = torch.zeros((1,), dtype=torch.int32, device=pages.device)
        self._r, self._r1 = (R,), (R + 1,)
        self._q_shape, self._o_shape = (R, cfg.num_q_heads, cfg.head_dim_qk), (R, cfg.num_q_heads, cfg.head_dim_v)
        self._prefix_sizes, self._evict_sizes = {}, {}
        self._scale = cfg.default_scale
        self._kv = _lib.hs_paged_kv(p, t, int(pages.shape[0]), int(pages.shape[1]), max_pages, self._err.data_ptr(),
                                    self.device)
        self._c_ref, self._kv_ref = ctypes.byref(self._c), ctypes.byref(self._kv)

    def _empty(self, shape, dtype, stream):
        """A tensor of this cache's device, allocated on the stream that uses it."""
        import torch

        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.pages.device)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self.pages.device)

    def append(self, k, v, cu, start, rope: RopeTable | None = None, rope_pos=None, q=None, q_out=None,
               rotary_offset: int | None = None, stream=None, q_weight=None, k_weight=None, eps: float = 1e-6):
        """Store the records of N new tokens, their keys (and queries) rotated by their positions.

        k bf16 [N][Hkv][Dqk], v bf16 [N][Hkv][Dv] (shared latent: k [N][Dqk], v None): views with any
        strides that are multiples of 16 bytes.  Tokens [cu[r], cu[r + 1]) (cu int32 [R + 1]) are request
        r's, stored from position start[r] (int64 [R]) on; tokens outside cu are padding.  rope_pos int64
        [N]: the positions whose angles they get, when not those they are stored at.  q bf16
        [N][Hq][Dqk] or [N][Hq][rotary_dim] -> q_out (may be q).  rotary_offset: first rotated value of a
        key; default 0, shared latent: the tail.  Returns q_out.

        With weights, heads are normed before they are rotated: x_i w_i / sqrt(mean(x^2) + eps).  q_weight, k_weight
        bf16 or float32 [Dqk], or [Hq][Dqk] and [Hkv][Dqk] for weights of each head; shared latent: k_weight [Dv], over the
        latent's values, no q_weight.  A table with axes takes rope_pos int64 [N][axes]."""
        import torch

        c = self.cfg
        if not isinstance(k, torch.Tensor) or k.dim() < 2:
            raise ValueError("k must be a tensor [N][Hkv][Dqk]")
        N, mla = int(k.shape[0]), c.layout == _lib.LAYOUT_MLA
        kp, kt, kh = _strided(torch, k, N, c.num_kv_heads, c.head_dim_qk, "k", self.device)
        vp, vt, vh = 0, 0, 0
        if mla != (v is None):
            raise ValueError("a shared latent has no v" if mla else "v is missing")
        if v is not None:
            vp, vt, vh = _strided(torch, v, N, c.num_kv_heads, c.head_dim_v, "v", self.device)
        cup = _fast_ptr(cu, torch.int32, self._r1, "cu", self.device)
        sp = _fast_ptr(start, torch.int64, self._r, "start", self.device)
        several = rope is not None and rope.axes > 1
        if several and rope_pos is None:
            raise ValueError("a rope with several axes needs rope_pos")
        rp = 0 if rope_pos is None else _fast_ptr(rope_pos, torch.int64, (N, rope.axes) if several else (N,), "rope_pos", self.device)
        turns, rd, il = 0, 0, 0
        if rope is not None:
            if rope.device != self.device:
                raise ValueError(f"rope must live on cuda:{self.device}")
            turns, rd, il = rope.turns.data_ptr(), rope.rotary_dim, int(rope.interleaved)
        if rotary_offset is None:
            rotary_offset = max(0, c.head_dim_qk - rd) if mla and rd else 0
        qp, qt, qh, op, ot, oh, qd = 0, 0, 0, 0, 0, 0, 0
        if q is not None:
            if not isinstance(q, torch.Tensor) or q.dim() != 3:
                raise ValueError("q must be a tensor [N][Hq][Dqk or rotary_dim]")
            qd = int(q.shape[2])
            if qd != c.head_dim_qk and (qd != rd or qd == 0):
                raise ValueError("the last dim of q must be head_dim_qk or rotary_dim")
            if q_out is None:
                q_out = self._empty((N, c.num_q_heads, qd), torch.bfloat16, stream)
            qp, qt, qh = _strided(torch, q, N, c.num_q_heads, qd, "q", self.device)
            op, ot, oh = _strided(torch, q_out, N, c.num_q_heads, qd, "q_out", self.device, written=True)
        elif q_out is not None:
            raise ValueError("q_out without q")
        normed = several or q_weight is not None or k_weight is not None
        if normed:
            b = self._norm_args(torch, c, mla, rope, q, qd, q_weight, k_weight, eps)
        a = _lib.pack_append.pack(N, cup, sp, rp, kp, kt, kh, vp, vt, vh, turns, rd, int(rotary_offset), il, qp, qt, qh, op, ot, oh, qd)
        if normed:
            _check("hs_append_normed", self.lib.hs_append_normed(self._c_ref, self._kv_ref, a, b, _fast_stream(torch, stream, self.device)))
        else:
            _check("hs_append_rotated", self.lib.hs_append_rotated(self._c_ref, self._kv_ref, a,
                                                                   _fast_stream(torch, stream, self.device)))
        return q_out

    def _norm_args(self, torch, c, mla, rope, q, qd, q_weight, k_weight, eps):
        """What hs_append_normed takes beside the arguments of hs_append_rotated, packed."""
        dim = c.head_dim_v if mla else c.head_dim_qk
        kw, ks, kt = _weights(torch, k_weight, c.num_kv_heads, dim, "k_weight", self.device)
        if q_weight is not None and (mla or q is None or qd != c.head_dim_qk):
            raise ValueError("q_weight needs whole query heads (and no shared latent)")
        qw, qs, qt = _weights(torch, q_weight, c.num_q_heads, dim, "q_weight", self.device)
        if (qw or kw) and not (0.0 < eps < float("inf")):
            raise ValueError("eps must be a positive number")
        axis = rope.axis if rope is not None else None
        return _lib.pack_norm.pack(kw, ks, qw, qs, kt, qt, float(eps), 1 if axis is None else rope.axes,
                                   0 if axis is None else axis.data_ptr())

    def evict(self, lens, weights, keep: int, first=0, recent: int = 0, weights_out=None, lens_out=None, stream=None):
        """Cut every request of more than `keep` entries down to that many: its first `first` and last `recent` entries and, of
        the others, those with the largest weights (of equal ones the earlier), in their order, become the entries [0, keep),
        records and weights alike.

        lens int64 [R]; weights float32 [R][lists][C], what prefix_attn sums up: lists 1 (a request's entries go together) or
        Hkv (each KV head keeps its own).  first: a number, or int64 [R] on the device (a shared prefix stays whole:
        pages of several requests must lie within it).  weights_out (default: weights, in place): the weights of what stays, 0
        behind it up to lens.  Returns lens_out, min(lens, keep) (default: a new tensor; may be lens).  Keys keep the
        rotation they were stored with: append the next tokens with rope_pos."""
        import torch

        c = self.cfg
        if not isinstance(weights, torch.Tensor) or weights.dim() != 3 or weights.shape[1] not in (1, c.num_kv_heads):
            raise ValueError("weights must be a tensor [R][1 or Hkv][C]")
        shape = (c.num_requests, int(weights.shape[1]), int(weights.shape[2]))
        lp = _fast_ptr(lens, torch.int64, self._r, "lens", self.device)
        wp = _fast_ptr(weights, torch.float32, shape, "weights", self.device)
        op = wp if weights_out is None else _fast_ptr(weights_out, torch.float32, shape, "weights_out", self.device)
        keep, recent = int(keep), int(recent)
        fp, f = 0, 0
        if isinstance(first, torch.Tensor):
            fp = _fast_ptr(first, torch.int64, self._r, "first", self.device)
        else:
            f = int(first)
        if not 1 <= keep <= 2**31 - 65536 or recent < 0 or f < 0 or f + recent > keep:
            raise ValueError("keep must be positive, first and recent together at most keep")
        need = self._evict_sizes.get((shape[1], keep))
        if need is None:
            need = int(self.lib.hs_evict_workspace(self._c_ref, shape[1], keep))
            if need < 0:
                raise HsError("hs_evict_workspace", need)
            self._evict_sizes[shape[1], keep] = need
        if lens_out is None:
            lens_out = self._empty(self._r, torch.int64, stream)
        ws = self._empty((need,), torch.uint8, stream)
        np_ = _fast_ptr(lens_out, torch.int64, self._r, "lens_out", self.device)
        a = _lib.pack_evict.pack(lp, wp, op, np_, fp, shape[2], shape[1], keep, f, recent, ws.data_ptr(), need)
        _check("hs_evict", self.lib.hs_evict(self._c_ref, self._kv_ref, a, _fast_stream(torch, stream, self.device)))
        return lens_out

    def tree_attn(self, q, lens, mask, locs=None, nodes=None, out=None, scale=None, stream=None):
        """Attention of T drafted tokens a request, stored at positions [lens[r], lens[r] + T), over the
        context and each other.  q bf16 [R][T][Hq][Dqk]; lens int64 [R]; mask int64 [R][T][ceil(T/64)]
        (see tree_mask); locs int32 [R][k]: only these positions of the context (-1 = padding), else all
        of [0, lens[r]); nodes int32 [R]: nodes in use, output rows behind them are left as they were.
        Returns out, bf16 [R][T][Hq][Dv] (it may not overlap q)."""
        import torch

        c = self.cfg
        lp, kp, k = _fast_ptr(lens, torch.int64, self._r, "lens", self.device), 0, 0
        if locs is not None:
            if locs.dim() != 2 or locs.shape[1] < 1:
                raise ValueError("locs must be [R][k] with k >= 1")
            k = locs.shape[1]
            kp = _fast_ptr(locs, torch.int32, (c.num_requests, k), "locs", self.device)
        args, out, _ws = _tree_args(torch, self.lib, self._c, c, self.device, self._tree_sizes, q, lp, kp, k, mask, nodes, out, scale,
                                    stream)
        _check("hs_tree_attn", self.lib.hs_tree_attn(self._c_ref, self._kv_ref, args, _fast_stream(torch, stream, self.device)))
        return out

    def prefix_attn(self, q, lens, groups=None, prefix=None, weights=None, decay: float = 1.0, out=None, scale=None, stream=None):
        """Attention of one new token a request over the positions [0, lens[r]), those that requests share read for many at a time.

        q bf16 [R][Hq][Dqk]; lens int64 [R], the new tokens' own positions among them.  groups int32 [G + 1]
        ascending and prefix int64 [G]: the requests [groups[g], groups[g + 1]) share the positions [0, prefix[g]), which
        are read through the table's row of the first of them; the other requests share none.  weights float32
        [R][lists][C], lists 1 or Hkv: takes weights * decay + the softmax weights, summed over the list's query heads, of the
        positions behind a request's prefix (what evict goes by); the call's workspace then holds 4 bytes for each request, query
        head and position of the table.  Returns out, bf16 [R][Hq][Dv] (it may not overlap q)."""
        import torch

        c = self.cfg
        bf16 = torch.bfloat16
        qp = _fast_ptr(q, bf16, self._q_shape, "q", self.device)
        lp = _fast_ptr(lens, torch.int64, self._r, "lens", self.device)
        if (groups is None) != (prefix is None):
            raise ValueError("groups and prefix go together")
        G, gp, pp = 0, 0, 0
        if groups is not None:
            if not isinstance(prefix, torch.Tensor) or prefix.dim() != 1 or prefix.shape[0] > c.num_requests:
                raise ValueError("prefix must be a tensor [G] of at most R numbers")
            G = prefix.shape[0]
            gp = _fast_ptr(groups, torch.int32, (G + 1,), "groups", self.device)
            pp = _fast_ptr(prefix, torch.int64, (G,), "prefix", self.device)
        wp, cap, lists = 0, 0, 0
        if weights is not None:
            if not isinstance(weights, torch.Tensor) or weights.dim() != 3 or weights.shape[1] not in (1, c.num_kv_heads):
                raise ValueError("weights must be a tensor [R][1 or Hkv][C]")
            lists, cap = weights.shape[1], weights.shape[2]
            wp = _fast_ptr(weights, torch.float32, (self._r[0], lists, cap), "weights", self.device)
            if not abs(decay) < float("inf"):
                raise ValueError("decay must be a finite number")
        need = self._prefix_sizes.get((G, wp != 0))
        if need is None:
            need = int(self.lib.hs_prefix_attn_workspace(self._c_ref, self._kv_ref, G, int(wp != 0)))
            if need < 0:
                raise HsError("hs_prefix_attn_workspace", need)
            self._prefix_sizes[G, wp != 0] = need
        s = self._scale
        if scale is not None:
            s = float(scale)
            if not abs(s) <= 2.35e38:  # times log2(e) it has to be a finite 32-bit number
                raise ValueError("scale must be a number of magnitude 2.35e38 at most")
        if out is None:
            out = self._empty(self._o_shape, bf16, stream)
        ws = self._empty((need,), torch.uint8, stream)
        op = _fast_ptr(out, bf16, self._o_shape, "out", self.device)
        a = _lib.pack_prefix.pack(qp, lp, gp, pp, G, s, wp, cap, lists, decay, op, ws.data_ptr(), need)
        _check("hs_prefix_attn", self.lib.hs_prefix_attn(self._c_ref, self._kv_ref, a, _fast_stream(torch, stream, self.device)))
        return out

    def debug_stall_next(self):
        """Test hook: this thread's next prefix_attn on the tensor cores has a barrier wait for an arrival that nothing makes, so its
        bounded waits give up and DEVERR_TIMEOUT is reported; its outputs are then undefined."""
        _check("hs_debug_stall_prefix", self.lib.hs_debug_stall_prefix())

    def keep_path(self, lens, path, count, stream=None):
        """The record of node path[r][i] moves to position lens[r] + i for i < count[r].  lens int64 [R];
        path int32 [R][P], ascending nodes; count int32 [R]."""
        import torch

        if not isinstance(path, torch.Tensor) or path.dim() != 2:
            raise ValueError("path must be a tensor [R][P]")
        P = path.shape[1]
        lp = _fast_ptr(lens, torch.int64, self._r, "lens", self.device)
        pp = _fast_ptr(path, torch.int32, (self._r[0], P), "path", self.device)
        cp = _fast_ptr(count, torch.int32, self._r, "count", self.device)
        _check("hs_keep_path", self.lib.hs_keep_path(self._c_ref, self._kv_ref, lp, pp, P, cp,
                                                     _fast_stream(torch, stream, self.device)))

    def errors(self, reset: bool = False) -> int:
        """The DEVERR_* bits that the calls so far recorded (synchronises the device).  DEVERR_TIMEOUT: a tree
        or prefix attention gave up waiting, its output and the weights it sums up are undefined; the cache is as it was."""
        import torch

        torch.cuda.synchronize(self.device)
        bits = int(self._err.item())
        if reset:
            self._err.zero_()
            torch.cuda.synchronize(self.device)
        return bits
