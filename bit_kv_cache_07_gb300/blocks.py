"""The block cache: requests of a serving batch share one pool of blocks of 32
tokens, held in 8 bits with one scale for each block, KV head and side (the
kvq_block calls of include/kvq.h).

``Tables`` holds what the layers of a model share and what changes from step to
step, all of it on the GPU; ``Layer`` one layer's codes and scales.  A step is

    tables.plan(n_new)                                   # once
    layer.append(tables, k, v, q, q, q_weight, k_weight) # per layer
    layer.attn(tables, q, out, lse, workspace)

and can be captured in a CUDA graph: lengths, tables and new tokens are read on
the GPU.  Arguments are checked before the call; nothing here computes.
"""
from __future__ import annotations

import ctypes as C

from .binding import (BLOCK_TABLES, KvqError, _arg, _check, _on_device, _stream_of, kvq_block_config, kvq_block_layout,
                      kvq_block_tables, lib)

BLOCK_TOKENS = 32
_SHARED = ("batch", "n_tokens", "n_blocks", "max_blocks")  # what tables and layers agree in


def make_config(d) -> kvq_block_config:
    """kvq_block_config from a dict with the same field names (missing -> 0)."""
    if isinstance(d, kvq_block_config):
        return d
    known = {n: t for n, t in kvq_block_config._fields_}
    for name in d:
        if name not in known:
            raise ValueError(f"no field {name!r} in a block cache's configuration")
    c = kvq_block_config()
    for name, t in known.items():
        if name in d:
            setattr(c, name, float(d[name]) if t is C.c_float else int(d[name]))
    return c


def layout(cfg) -> kvq_block_layout:
    """Bytes of a layer's codes and scales and of the attention's scratch."""
    out = kvq_block_layout()
    _check("kvq_block_layout_query", lib().kvq_block_layout_query(C.byref(make_config(cfg)), C.byref(out)))
    return out


def new_workspace(cfg, device="cuda"):
    """Zeroed scratch for ``Layer.attn``."""
    import torch
    return torch.zeros(layout(cfg).workspace_bytes, dtype=torch.uint8, device=device)


def _ints(t, what: str, shape):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != shape:
        raise ValueError(f"{what}: expected a contiguous int32 CUDA tensor of shape {shape}")
    return t.data_ptr()


class Tables:
    """Block tables, the free stack, lengths and the step's offsets and slot maps,
    shared by the layers of a model; every block is free and every request empty
    unless tensors of the layout of kvq_block_tables are given by name."""

    def __init__(self, cfg, device="cuda", **arrays):
        import torch
        self.cfg = make_config(cfg)
        layout(self.cfg)  # its refusals
        c = self.cfg
        self.shared = tuple(getattr(c, n) for n in _SHARED)
        shapes = dict(block_table=(c.batch, c.max_blocks), free_list=(c.n_blocks,), free_count=(1,), lens=(c.batch,),
                      start=(c.batch + 1,), unit0=(c.batch + 1,), token_row=(c.n_tokens,), position=(c.n_tokens,),
                      slot=(c.n_tokens,))
        for name in arrays:
            if name not in shapes:
                raise ValueError(f"no array {name!r} in a block cache's tables")
        for name in BLOCK_TABLES:
            t = arrays.get(name)
            if t is None:
                if name == "free_list":  # the lowest block on top
                    t = torch.arange(c.n_blocks - 1, -1, -1, dtype=torch.int32, device=device)
                elif name == "free_count":
                    t = torch.full((1,), c.n_blocks, dtype=torch.int32, device=device)
                else:
                    t = torch.zeros(shapes[name], dtype=torch.int32, device=device)
            setattr(self, name, t)
        self.arrays = kvq_block_tables(*[_ints(getattr(self, n), n, shapes[n]) for n in BLOCK_TABLES])
        self._refs = C.byref(self.cfg), C.byref(self.arrays)
        if len({getattr(self, n).device for n in BLOCK_TABLES}) != 1:
            raise ValueError("the tables must be on one device")

    def plan(self, n_new, lens=None, free_count=None, stream=None):
        """The step's tables: request b adds n_new[b] tokens, or ends (negative).
        lens, free_count: lengths and free blocks before the step, the tables' own
        (updated in place) unless given."""
        rows = (self.cfg.batch,)
        np_ = _ints(n_new, "n_new", rows)
        lp = self.arrays.lens if lens is None else _ints(lens, "lens", rows)
        fp = self.arrays.free_count if free_count is None else _ints(free_count, "free_count", (1,))
        _on_device(self.lens, n_new, lens, free_count)
        _check("kvq_block_plan", lib().kvq_block_plan(*self._refs, lp, fp, np_, _stream_of(stream, self.lens)))


def _rows(t, what: str, tokens: int, heads: int):
    """(address, elements from a token to the next) of fp16 rows [tokens, heads, 128]
    whose heads lie one after the other."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float16 or not t.is_cuda or tuple(t.shape) != (tokens, heads, 128):
        raise ValueError(f"{what}: expected a float16 CUDA tensor of shape {(tokens, heads, 128)}")
    s = t.stride()
    if s[2] != 1 or (heads > 1 and s[1] != 128):
        raise ValueError(f"{what}: a token's heads must lie one after the other")
    return t.data_ptr(), s[0] if tokens > 1 else heads * 128


def _weight(t, what: str):
    import torch
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or tuple(t.shape) != (128,):
        raise ValueError(f"{what}: expected a tensor of shape (128,)")
    return _arg(t, what, torch.float16, 256)


class Layer:
    """One layer's cache: zeroed codes uint8 [n_blocks, Hkv, 2, 32, 128] and scales
    uint8 [n_blocks, Hkv, 2], or tensors of that layout."""

    def __init__(self, cfg, codes=None, scales=None, device="cuda"):
        import torch
        self.cfg = make_config(cfg)
        self.layout = layout(self.cfg)
        c = self.cfg
        self.shared = tuple(getattr(c, n) for n in _SHARED)
        shape = (c.n_blocks, c.n_kv_heads, 2)
        if codes is None:
            codes = torch.zeros(shape + (BLOCK_TOKENS, 128), dtype=torch.uint8, device=device)
        if scales is None:
            room = torch.zeros(self.layout.scales_bytes, dtype=torch.uint8, device=device)
            scales = room[:c.n_blocks * c.n_kv_heads * 2].view(shape)
        self._codes = _arg(codes, "codes", torch.uint8, self.layout.codes_bytes)
        self._scales = _arg(scales, "scales", torch.uint8, c.n_blocks * c.n_kv_heads * 2)
        if tuple(codes.shape) != shape + (BLOCK_TOKENS, 128) or tuple(scales.shape) != shape:
            raise ValueError(f"codes, scales: expected shapes {shape + (BLOCK_TOKENS, 128)} and {shape}")
        if scales.untyped_storage().nbytes() - scales.storage_offset() < self.layout.scales_bytes:
            raise ValueError(f"scales: its storage must reach {self.layout.scales_bytes} bytes (padded to 16)")
        if codes.device != scales.device:
            raise ValueError("codes and scales must be on one device")
        self.codes, self.scales = codes, scales
        self._ref = C.byref(self.cfg)

    def _tables(self, tables):
        if tables.shared != self.shared:
            raise ValueError(f"tables and layer differ in {', '.join(_SHARED)}: {tables.shared}, {self.shared}")
        return tables._refs[1]

    def append(self, tables: Tables, k, v, q=None, q_out=None, q_weight=None, k_weight=None, stream=None):
        """The planned tokens' keys and values [n_tokens, Hkv, 128] into the blocks,
        and the queries [n_tokens, Hq, 128] normed and rotated into q_out (q itself,
        or apart from it).  k, v, q may be parts of one projection's rows."""
        c = self.cfg
        tp = self._tables(tables)
        kp, ks = _rows(k, "k", c.n_tokens, c.n_kv_heads)
        vp, vs = _rows(v, "v", c.n_tokens, c.n_kv_heads)
        qp = op = None
        qs = 0
        if q is not None or q_out is not None:
            if q is None or q_out is None:
                raise ValueError("q and q_out go together")
            qp, qs = _rows(q, "q", c.n_tokens, c.n_q_heads)
            op, os_ = _rows(q_out, "q_out", c.n_tokens, c.n_q_heads)
            if os_ != c.n_q_heads * 128:
                raise ValueError("q_out must be contiguous")
        _on_device(tables.lens, self.codes, k, v, q, q_out, q_weight, k_weight)
        _check("kvq_block_append", lib().kvq_block_append(
            self._ref, tp, self._codes, self._scales, kp, ks, vp, vs, qp, qs, op, _weight(q_weight, "q_weight"),
            _weight(k_weight, "k_weight"), _stream_of(stream, k)))

    def attn(self, tables: Tables, q, out, lse=None, workspace=None, stream=None):
        """Attention of the planned tokens' queries [n_tokens, Hq, 128] (as append
        leaves them) over their requests' blocks into out, and the log-sum-exp
        [n_tokens, Hq] into lse."""
        import torch
        c = self.cfg
        tp = self._tables(tables)
        qp, qs = _rows(q, "q", c.n_tokens, c.n_q_heads)
        op, os_ = _rows(out, "out", c.n_tokens, c.n_q_heads)
        if qs != c.n_q_heads * 128 or os_ != qs:
            raise ValueError("q and out must be contiguous")
        lp = None
        if lse is not None:
            lp = _arg(lse, "lse", torch.float32, 4 * c.n_tokens * c.n_q_heads)
            if tuple(lse.shape) != (c.n_tokens, c.n_q_heads):
                raise ValueError(f"lse: expected shape {(c.n_tokens, c.n_q_heads)}, got {tuple(lse.shape)}")
        if workspace is None:
            raise KvqError("kvq_block_attn", -4)
        wp = _arg(workspace, "workspace", torch.uint8, 0)
        _on_device(tables.lens, self.codes, q, out, lse, workspace)
        _check("kvq_block_attn", lib().kvq_block_attn(self._ref, tp, self._codes, self._scales, qp, op, lp, wp,
                                                     workspace.nbytes, _stream_of(stream, q)))
