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

import torch

from .binding import (BLOCK_TABLES, KvqError, _check, kvq_block_config, kvq_block_layout, kvq_block_tables, lib)

BLOCK_TOKENS = 32
_SHARED = ("batch", "n_tokens", "n_blocks", "max_blocks")  # what tables and layers agree in


def make_config(d) -> kvq_block_config:
    """kvq_block_config from a dict with the same field names (missing -> 0), or a
    copy of one: what tables and layers hold agrees with their arrays, whatever the
    caller writes into the configuration afterwards."""
    if isinstance(d, kvq_block_config):
        return kvq_block_config.from_buffer_copy(d)
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
    return torch.zeros(layout(cfg).workspace_bytes, dtype=torch.uint8, device=device)


def _here() -> int:
    """The device that the calls launch on: the current one; their tensors live there."""
    return torch._C._cuda_getDevice()


def _stream_on(stream, device: int):
    """A stream's handle; None: the device's current stream."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _refuse(t, what: str, dtype, shape, device):
    """The error for a tensor that is not of this type and shape on this device."""
    want = f"{what}: expected a {dtype} tensor of shape {tuple(shape)} on cuda:{device}"
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{want}, got {type(t).__name__}")
    raise ValueError(f"{want}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _dense(t, what: str, dtype, shape, device) -> int:
    """The address of a contiguous tensor."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == device:
        raise ValueError(f"{what} must be contiguous")
    _refuse(t, what, dtype, shape, device)


def _ints(t, what: str, shape, device) -> int:
    return _dense(t, what, torch.int32, shape, device)


def _kept(name):
    """An attribute whose tensor's address the kernels hold: written in place, never
    exchanged (the calls would go on with the old one's memory)."""
    def put(self, value):
        if value is not self._tensors[name]:  # (`x.lens += 1` assigns the tensor itself)
            raise AttributeError(f"{name}: the calls hold the address of its tensor; write into it in place")
    return property(lambda self: self._tensors[name], put)


class Tables:
    """Block tables, the free stack, lengths and the step's offsets and slot maps,
    shared by the layers of a model; every block is free and every request empty
    unless tensors of the layout of kvq_block_tables are given by name.  They are
    attributes of these names and are written in place."""

    cfg = property(lambda self: make_config(self._cfg), doc="a copy of the configuration")
    block_table, free_list, free_count, lens, start, unit0, token_row, position, slot = map(_kept, BLOCK_TABLES)

    def __init__(self, cfg, device="cuda", **arrays):
        self._cfg = make_config(cfg)
        layout(self._cfg)  # its refusals
        c = self._cfg
        self.shared = tuple(getattr(c, n) for n in _SHARED)
        shapes = dict(block_table=(c.batch, c.max_blocks), free_list=(c.n_blocks,), free_count=(1,), lens=(c.batch,),
                      start=(c.batch + 1,), unit0=(c.batch + 1,), token_row=(c.n_tokens,), position=(c.n_tokens,),
                      slot=(c.n_tokens,))
        for name in arrays:
            if name not in shapes:
                raise ValueError(f"no array {name!r} in a block cache's tables")
        self._tensors = {}
        for name in BLOCK_TABLES:
            t = arrays.get(name)
            if t is None:
                if name == "free_list":  # the lowest block on top
                    t = torch.arange(c.n_blocks - 1, -1, -1, dtype=torch.int32, device=device)
                elif name == "free_count":
                    t = torch.full((1,), c.n_blocks, dtype=torch.int32, device=device)
                else:
                    t = torch.zeros(shapes[name], dtype=torch.int32, device=device)
            self._tensors[name] = t
        self.device = self.lens.get_device() if isinstance(self.lens, torch.Tensor) else None
        self.arrays = kvq_block_tables(*[_ints(t, n, shapes[n], self.device) for n, t in self._tensors.items()])
        if self.device < 0:
            raise ValueError("the tables must be on a GPU")
        self._refs = C.byref(self._cfg), C.byref(self.arrays)
        self._call, self._call_back = lib().kvq_block_plan, lib().kvq_block_plan_back
        self._rows = (c.batch,)

    def plan(self, n_new, lens=None, free_count=None, stream=None, n_back=None):
        """The step's tables: request b adds n_new[b] tokens, or ends (negative).
        lens, free_count: lengths and free blocks before the step, the tables' own
        (updated in place) unless given.  n_back: tokens that a request takes back
        first (drafted ones that were not accepted); lengths are lowered in no other
        way, or the blocks behind them are lost."""
        d = _here()
        if d != self.device:
            raise ValueError(f"the tables are on cuda:{self.device}, the current device is cuda:{d}")
        np_ = _ints(n_new, "n_new", self._rows, d)
        lp = self.arrays.lens if lens is None else _ints(lens, "lens", self._rows, d)
        fp = self.arrays.free_count if free_count is None else _ints(free_count, "free_count", (1,), d)
        if n_back is None:
            st = self._call(*self._refs, lp, fp, np_, _stream_on(stream, d))
        else:
            st = self._call_back(*self._refs, lp, fp, np_, _ints(n_back, "n_back", self._rows, d), _stream_on(stream, d))
        if st:
            _check("kvq_block_plan", st)


def _strided(t, what: str, shape, dense, device):
    """(address, elements from a token to the next) of fp16 rows [tokens, heads, 128]
    whose heads lie one after the other; dense: the strides of contiguous ones."""
    try:
        if t.dtype is torch.float16 and t.shape == shape and t.get_device() == device:
            s = t.stride()
            if s == dense:
                return t.data_ptr(), dense[0]
            if s[2] == 1 and (s[1] == 128 or shape[1] == 1):
                return t.data_ptr(), s[0] if shape[0] > 1 else dense[0]
            raise ValueError(f"{what}: a token's heads must lie one after the other")
    except AttributeError:
        pass
    _refuse(t, what, torch.float16, shape, device)


class Layer:
    """One layer's cache: zeroed codes uint8 [n_blocks, Hkv, 2, 32, 128] and scales
    uint8 [n_blocks, Hkv, 2], or tensors of that layout."""

    cfg = property(lambda self: make_config(self._cfg), doc="a copy of the configuration")
    codes, scales = map(_kept, ("codes", "scales"))

    def __init__(self, cfg, codes=None, scales=None, device="cuda"):
        self._cfg = make_config(cfg)
        self.layout = layout(self._cfg)
        c = self._cfg
        self.shared = tuple(getattr(c, n) for n in _SHARED)
        shape = (c.n_blocks, c.n_kv_heads, 2)
        if codes is None:
            codes = torch.zeros(shape + (BLOCK_TOKENS, 128), dtype=torch.uint8, device=device)
        if scales is None:
            room = torch.zeros(self.layout.scales_bytes, dtype=torch.uint8, device=device)
            scales = room[:c.n_blocks * c.n_kv_heads * 2].view(shape)
        self.device = codes.get_device() if isinstance(codes, torch.Tensor) else None
        self._codes = _dense(codes, "codes", torch.uint8, shape + (BLOCK_TOKENS, 128), self.device)
        self._scales = _dense(scales, "scales", torch.uint8, shape, self.device)
        if self.device < 0:
            raise ValueError("codes and scales must be on a GPU")
        if scales.untyped_storage().nbytes() - scales.storage_offset() < self.layout.scales_bytes:
            raise ValueError(f"scales: its storage must reach {self.layout.scales_bytes} bytes (padded to 16)")
        self._tensors = dict(codes=codes, scales=scales)
        self._ref = C.byref(self._cfg)
        self._append, self._attn = lib().kvq_block_append, lib().kvq_block_attn
        self._kv = (c.n_tokens, c.n_kv_heads, 128), (c.n_kv_heads * 128, 128, 1)
        self._q = (c.n_tokens, c.n_q_heads, 128), (c.n_q_heads * 128, 128, 1)
        self._lse = (c.n_tokens, c.n_q_heads)

    def _ready(self, tables):
        """The current device, which the layer and the tables must be on."""
        if tables.shared != self.shared:
            raise ValueError(f"tables and layer differ in {', '.join(_SHARED)}: {tables.shared}, {self.shared}")
        d = _here()
        if d != self.device or d != tables.device:
            raise ValueError(f"the layer is on cuda:{self.device}, the tables on cuda:{tables.device}, the current device is cuda:{d}")
        return d

    def append(self, tables: Tables, k, v, q=None, q_out=None, q_weight=None, k_weight=None, stream=None):
        """The planned tokens' keys and values [n_tokens, Hkv, 128] into the blocks,
        and the queries [n_tokens, Hq, 128] normed and rotated into q_out (q itself,
        or apart from it).  k, v, q may be parts of one projection's rows."""
        d = self._ready(tables)
        kp, ks = _strided(k, "k", *self._kv, d)
        vp, vs = _strided(v, "v", *self._kv, d)
        qp = op = wq = wk = None
        qs = 0
        if q is not None or q_out is not None:
            if q is None or q_out is None:
                raise ValueError("q and q_out go together")
            qp, qs = _strided(q, "q", *self._q, d)
            op = _dense(q_out, "q_out", torch.float16, self._q[0], d)
        if q_weight is not None:
            wq = _dense(q_weight, "q_weight", torch.float16, (128,), d)
        if k_weight is not None:
            wk = _dense(k_weight, "k_weight", torch.float16, (128,), d)
        st = self._append(self._ref, tables._refs[1], self._codes, self._scales, kp, ks, vp, vs, qp, qs, op, wq, wk, _stream_on(stream, d))
        if st:
            _check("kvq_block_append", st)

    def attn(self, tables: Tables, q, out, lse=None, workspace=None, stream=None):
        """Attention of the planned tokens' queries [n_tokens, Hq, 128] (as append
        leaves them) over their requests' blocks into out, and the log-sum-exp
        [n_tokens, Hq] into lse."""
        d = self._ready(tables)
        qp = _dense(q, "q", torch.float16, self._q[0], d)
        op = _dense(out, "out", torch.float16, self._q[0], d)
        lp = None if lse is None else _dense(lse, "lse", torch.float32, self._lse, d)
        if workspace is None:
            raise KvqError("kvq_block_attn", -4)
        if not isinstance(workspace, torch.Tensor):
            raise ValueError(f"workspace: expected a uint8 tensor on cuda:{d}, got {type(workspace).__name__}")
        wp = _dense(workspace, "workspace", torch.uint8, workspace.shape, d)
        st = self._attn(self._ref, tables._refs[1], self._codes, self._scales, qp, op, lp, wp, workspace.nbytes, _stream_on(stream, d))
        if st:
            _check("kvq_block_attn", st)
