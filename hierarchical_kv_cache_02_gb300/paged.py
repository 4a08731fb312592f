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
from .pool import HsConfig, _check, _dev_tensor, _fast_ptr, _fast_stream, _tree_args


class RopeTable:
    """Frequencies of a rotary embedding on one device, as fractions of a turn per position.

    rotary_dim: rotated values of a head, a multiple of 16.  inv_freq: rotary_dim / 2 angles per position
    (radians); default theta ** (-2 j / rotary_dim).  interleaved: value 2j turns with 2j + 1, else j with
    j + rotary_dim / 2."""

    def __init__(self, rotary_dim: int, theta: float = 10000.0, inv_freq=None, interleaved: bool = False,
                 device: int = 0):
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
        self.turns = torch.from_numpy(turns.view(np.int64)).to(f"cuda:{self.device}")


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


def _strided(t, n, heads, dim, name, device, written=False):
    """Pointer, token stride and head stride of a bf16 [n][heads][dim] view ([n][dim] when heads is 1)."""
    import torch

    if isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.shape == (n, heads, dim) and t.get_device() == device:
        ts, hs, vs = t.stride()
        p = t.data_ptr()
        if vs == 1 and n > 1 and heads > 1 and not (ts | hs | p >> 1) & 7 and (not written or ts >= (heads - 1) * hs + dim):
            return p, ts, hs  # what most calls pass; the rest is looked at one by one

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
        self._kv = _lib.hs_paged_kv(p, t, int(pages.shape[0]), int(pages.shape[1]), max_pages, self._err.data_ptr(),
                                    self.device)
        self._c_ref, self._kv_ref = ctypes.byref(self._c), ctypes.byref(self._kv)

    def append(self, k, v, cu, start, rope: RopeTable | None = None, rope_pos=None, q=None, q_out=None,
               rotary_offset: int | None = None, stream=None):
        """Store the records of N new tokens, their keys (and queries) rotated by their positions.

        k bf16 [N][Hkv][Dqk], v bf16 [N][Hkv][Dv] (shared latent: k [N][Dqk], v None): views with any
        strides that are multiples of 16 bytes.  Tokens [cu[r], cu[r + 1]) (cu int32 [R + 1]) are request
        r's, stored from position start[r] (int64 [R]) on; tokens outside cu are padding.  rope_pos int64
        [N]: the positions whose angles they get, when not those they are stored at.  q bf16
        [N][Hq][Dqk] or [N][Hq][rotary_dim] -> q_out (may be q).  rotary_offset: first rotated value of a
        key; default 0, shared latent: the tail.  Returns q_out."""
        import torch

        c = self.cfg
        if not isinstance(k, torch.Tensor) or k.dim() < 2:
            raise ValueError("k must be a tensor [N][Hkv][Dqk]")
        N, mla = int(k.shape[0]), c.layout == _lib.LAYOUT_MLA
        kp, kt, kh = _strided(k, N, c.num_kv_heads, c.head_dim_qk, "k", self.device)
        vp, vt, vh = 0, 0, 0
        if mla != (v is None):
            raise ValueError("a shared latent has no v" if mla else "v is missing")
        if v is not None:
            vp, vt, vh = _strided(v, N, c.num_kv_heads, c.head_dim_v, "v", self.device)
        cup = _fast_ptr(cu, torch.int32, self._r1, "cu", self.device)
        sp = _fast_ptr(start, torch.int64, self._r, "start", self.device)
        rp = 0 if rope_pos is None else _fast_ptr(rope_pos, torch.int64, (N,), "rope_pos", self.device)
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
                with torch.cuda.stream(stream):  # None: the current one
                    q_out = torch.empty((N, c.num_q_heads, qd), dtype=torch.bfloat16, device=q.device)
            qp, qt, qh = _strided(q, N, c.num_q_heads, qd, "q", self.device)
            op, ot, oh = _strided(q_out, N, c.num_q_heads, qd, "q_out", self.device, written=True)
        elif q_out is not None:
            raise ValueError("q_out without q")
        a = _lib.pack_append.pack(N, cup, sp, rp, kp, kt, kh, vp, vt, vh, turns, rd, int(rotary_offset), il, qp, qt, qh, op, ot, oh, qd)
        _check("hs_append_rotated", self.lib.hs_append_rotated(self._c_ref, self._kv_ref, a,
                                                               _fast_stream(torch, stream, self.device)))
        return q_out

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
        attention gave up waiting and its output is undefined; the cache is as it was."""
        import torch

        torch.cuda.synchronize(self.device)
        bits = int(self._err.item())
        if reset:
            self._err.zero_()
            torch.cuda.synchronize(self.device)
        return bits
