"""qwen3_vl_decoder_b200: the Qwen3-VL text decoder on B200 (sm_100a).

The full-sequence causal prefill of a layer or a stack, a KV cache written by
the prefill with one-token decode against it, and the steps either side: the
token-embedding gather with the soft-token splice, and the final norm + LM head.
For serving in 8 bits: a norm and a weight form with e4m3 outputs, their product,
and a cache of half the bytes with the attention that reads it.

A thin torch-facing binding of libq3vl's C ABI (include/q3vl.h). torch only
provides device memory and the current stream; every step runs in the
library's CUDA kernels, and there is no other implementation to fall back
to: without the built library, the first call raises ImportError.
"""
from __future__ import annotations

import ctypes
from typing import Dict, List, Optional, Sequence, Tuple, Union

import torch

from . import _abi
from ._abi import (Config, KvCache as KvCacheStruct, KvCacheQ8 as KvCacheQ8Struct,  # noqa: F401
                   Layer, RawWeights)

_lib_handle: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """The loaded libq3vl (loaded on first use; raises ImportError if not built)."""
    global _lib_handle
    if _lib_handle is None:
        _lib_handle = _abi.load()
    return _lib_handle

RAW_NAMES = ("attn_norm", "wq", "wk", "wv", "bq", "bk", "bv", "q_norm", "k_norm", "wo",
             "ffn_norm", "wg", "wu", "wd")


class Q3VLError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{_abi.STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


def version() -> str:
    return lib().q3vl_version().decode()


def _check(rc: int) -> None:
    if rc != _abi.OK:
        raise Q3VLError(rc, lib().q3vl_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The current device and its current stream's handle, by the functions below torch.cuda's where this
# torch has them (no Stream object is built: 3 us a call).
_device = getattr(torch._C, "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())
_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None) or
               (lambda index: torch.cuda.current_stream(index).cuda_stream))


def _stream(stream=None):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    if not torch.cuda.is_initialized():
        torch.cuda.init()
    return ctypes.c_void_p(_raw_stream(_device()))


def config(hidden, n_heads, n_kv_heads, intermediate, dtype="bf16", qkv_bias=False,
           head_dim=128, rope_theta=5e6, rms_eps=1e-6, mrope_section=(24, 20, 20)) -> Config:
    c = Config()
    c.hidden, c.n_heads, c.n_kv_heads, c.head_dim = hidden, n_heads, n_kv_heads, head_dim
    c.intermediate = intermediate
    c.dtype = _abi.DTYPE_BF16 if dtype == "bf16" else _abi.DTYPE_FP32
    c.has_qkv_bias = int(bool(qkv_bias))
    c.mrope_section[:] = list(mrope_section)
    c.rope_theta, c.rms_eps = float(rope_theta), float(rms_eps)
    return c


def config_of(w) -> Config:
    """Config of a q3vl_synth.Workload (or any object with the same fields)."""
    return config(w.hidden, w.n_heads, w.n_kv_heads, w.intermediate, w.dtype, w.qkv_bias,
                  w.head_dim, w.rope_theta, w.rms_eps, w.mrope_section)


def torch_dtype(cfg: Config) -> torch.dtype:
    return torch.bfloat16 if cfg.dtype == _abi.DTYPE_BF16 else torch.float32


class PackedLayer:
    """A packed layer: the device buffer plus the views the library reads."""

    def __init__(self, buf: torch.Tensor, views: Layer):
        self.buf = buf
        self.views = views


def packed_layer_bytes(cfg: Config) -> int:
    return int(lib().q3vl_packed_layer_bytes(ctypes.byref(cfg)))


def pack_layer(cfg: Config, raw: Dict[str, torch.Tensor], stream=None) -> PackedLayer:
    """Packs raw layer weights (device tensors in the config dtype)."""
    n = packed_layer_bytes(cfg)
    if n == 0:
        _check(_abi.EINVAL)
    dev = raw["wq"].device
    buf = torch.empty(n, dtype=torch.uint8, device=dev)
    rw = RawWeights()
    for name in RAW_NAMES:
        t = raw.get(name)
        if t is not None:
            assert t.is_contiguous() and t.dtype == torch_dtype(cfg), name
        setattr(rw, name, None if t is None else t.data_ptr())
    views = Layer()
    _check(lib().q3vl_pack_layer(ctypes.byref(cfg), ctypes.byref(rw), _ptr(buf), n,
                                ctypes.byref(views), _stream(stream)))
    return PackedLayer(buf, views)


def mrope_positions(token_types: torch.Tensor, grids: Optional[torch.Tensor], stream=None,
                    check: bool = True):
    """P0: (t, h, w) positions [3, S] int32 and the next position.

    token_types: device uint8 [S] (0 text, 1 image); grids: device int32
    [n, 3] (t, merged rows, merged cols) or None. With ``check`` the call
    synchronises and raises on a grid/run mismatch.
    """
    S = token_types.numel()
    dev = token_types.device
    pos = torch.empty((3, S), dtype=torch.int32, device=dev)
    info = torch.empty(2, dtype=torch.int32, device=dev)
    n = 0 if grids is None else grids.shape[0]
    _check(lib().q3vl_mrope_positions(_ptr(token_types), S, _ptr(grids) if n else None, n,
                                     _ptr(pos), _ptr(info), _stream(stream)))
    if not check:
        return pos, info
    st, nxt = (int(v) for v in info.cpu())
    if st != _abi.OK:
        raise Q3VLError(st, "image placeholders and grids disagree")
    return pos, nxt


def workspace_bytes(cfg: Config, S: int) -> int:
    return int(lib().q3vl_workspace_bytes(ctypes.byref(cfg), S))


def workspace(cfg: Config, S: int, device="cuda") -> torch.Tensor:
    n = workspace_bytes(cfg, S)
    if n == 0:
        _check(_abi.EINVAL)
    return torch.empty(n, dtype=torch.uint8, device=device)


def layer_prefill(cfg: Config, layer: PackedLayer, x: torch.Tensor, pos: torch.Tensor,
                  ds_slab: Optional[torch.Tensor] = None, ds_rows: Optional[torch.Tensor] = None,
                  ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One decoder layer in place on x [S, H]; returns x."""
    S = x.shape[0]
    ws = workspace(cfg, S, x.device) if ws is None else ws
    n_img = 0 if ds_rows is None else ds_rows.numel()
    _check(lib().q3vl_layer_prefill(ctypes.byref(cfg), ctypes.byref(layer.views), _ptr(x), S,
                                   _ptr(pos), _ptr(ds_slab), _ptr(ds_rows), n_img, _ptr(ws),
                                   ws.numel(), _stream(stream)))
    return x


def layer_prefill_noalloc(cfg: Config, layer: PackedLayer, x: torch.Tensor, pos: torch.Tensor,
                          ds_slab: Optional[torch.Tensor] = None,
                          ds_rows: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """layer_prefill with the library's built-in 64 MiB scratch instead of a workspace,
    for callers that cannot allocate device memory; calls must not overlap."""
    n_img = 0 if ds_rows is None else ds_rows.numel()
    _check(lib().q3vl_layer_prefill_noalloc(ctypes.byref(cfg), ctypes.byref(layer.views), _ptr(x),
                                            x.shape[0], _ptr(pos), _ptr(ds_slab), _ptr(ds_rows),
                                            n_img, _stream(stream)))
    return x


def stack_prefill(cfg: Config, layers: Sequence[PackedLayer], x: torch.Tensor, pos: torch.Tensor,
                  final_norm: Optional[torch.Tensor] = None,
                  ds_slabs: Sequence[torch.Tensor] = (), ds_rows: Optional[torch.Tensor] = None,
                  ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """n layers, DeepStack, optional final norm, in place on x; returns x."""
    S = x.shape[0]
    ws = workspace(cfg, S, x.device) if ws is None else ws
    arr = (Layer * len(layers))(*[l.views for l in layers])
    slabs = (ctypes.c_void_p * max(1, len(ds_slabs)))(*[s.data_ptr() for s in ds_slabs])
    n_img = 0 if ds_rows is None else ds_rows.numel()
    _check(lib().q3vl_stack_prefill(ctypes.byref(cfg), len(layers), arr, _ptr(final_norm), _ptr(x),
                                   S, _ptr(pos), slabs if ds_slabs else None, len(ds_slabs),
                                   _ptr(ds_rows), n_img, _ptr(ws), ws.numel(), _stream(stream)))
    return x


# ---------------------------------------------------------------------------
# KV cache and one-token decode (bf16)
# ---------------------------------------------------------------------------
Q8_BLOCK = 128   # columns, weight rows or tokens that share a scale


class KvCache:
    """One layer's cache: k and v bf16 [n_seq, cap, nkv*128] on the device (K after the
    per-head norm and MRoPE, as the prefill forms it)."""

    def __init__(self, cfg: Config, n_seq: int, cap: int, device="cuda"):
        dkv = cfg.n_kv_heads * cfg.head_dim
        self.k = torch.zeros((n_seq, cap, dkv), dtype=torch.bfloat16, device=device)
        self.v = torch.zeros_like(self.k)
        self.struct = KvCacheStruct(self.k.data_ptr(), self.v.data_ptr(), cap, n_seq)

    @property
    def cap(self) -> int:
        return int(self.struct.cap)


class KvCacheQ8:
    """One layer's 8-bit cache: k and v e4m3 [n_seq, cap, nkv*128] with E8M0 scales k_scale
    and v_scale [n_seq, ceil(cap/128), nkv], one per 128 tokens and KV head."""

    def __init__(self, cfg: Config, n_seq: int, cap: int, device="cuda"):
        dkv = cfg.n_kv_heads * cfg.head_dim
        blocks = -(-cap // Q8_BLOCK)

        def zeros(*shape):
            return torch.zeros(shape, dtype=torch.uint8, device=device)

        self._set(cfg, zeros(n_seq, cap, dkv).view(torch.float8_e4m3fn),
                  zeros(n_seq, cap, dkv).view(torch.float8_e4m3fn),
                  zeros(n_seq, blocks, cfg.n_kv_heads).view(torch.float8_e8m0fnu),
                  zeros(n_seq, blocks, cfg.n_kv_heads).view(torch.float8_e8m0fnu))

    @classmethod
    def of(cls, cfg: Config, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor,
           v_scale: torch.Tensor) -> "KvCacheQ8":
        """A cache over tensors that the caller holds already (kept, not copied)."""
        kv = cls.__new__(cls)
        kv._set(cfg, k, v, k_scale, v_scale)
        return kv

    def _set(self, cfg, k, v, k_scale, v_scale):
        _arg(k, "k", (torch.float8_e4m3fn,))
        if k.dim() != 3:
            raise Q3VLError(_abi.EINVAL, f"k must be [n_seq, cap, nkv*128], not {tuple(k.shape)}")
        n_seq, cap, dkv = k.shape
        blocks = -(-cap // Q8_BLOCK)
        for t, name in ((k, "k"), (v, "v")):
            _arg(t, name, (torch.float8_e4m3fn,), (n_seq, cap, cfg.n_kv_heads * cfg.head_dim),
                 k.device)
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _arg(t, name, (torch.float8_e8m0fnu,), (n_seq, blocks, cfg.n_kv_heads), k.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.struct = KvCacheQ8Struct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
                                      v_scale.data_ptr(), cap, n_seq)
        self.cap, self._width, self._index = cap, dkv, k.get_device()


def kv_caches(cfg: Config, n_layers: int, n_seq: int, cap: int, device="cuda",
              dtype="bf16") -> List[Union[KvCache, "KvCacheQ8"]]:
    """Caches of n_layers layers; dtype "bf16", or "fp8" for KvCacheQ8."""
    if dtype not in ("bf16", "fp8"):
        raise Q3VLError(_abi.EUNSUPPORTED, f"cache dtype must be 'bf16' or 'fp8', not {dtype!r}")
    cls = KvCache if dtype == "bf16" else KvCacheQ8
    return [cls(cfg, n_seq, cap, device) for _ in range(n_layers)]


def _is_q8(kvs: Sequence[Union[KvCache, KvCacheQ8]]) -> bool:
    """Whether the layers' caches are 8-bit; all of them have to be of one kind."""
    q8 = [isinstance(kv, KvCacheQ8) for kv in kvs]
    if any(q8) and not all(q8):
        raise Q3VLError(_abi.EINVAL, "the layers' caches must be all bf16 or all 8-bit")
    return any(q8)


def _kv_array(kvs: Sequence[Union[KvCache, KvCacheQ8]]):
    struct = KvCacheQ8Struct if _is_q8(kvs) else KvCacheStruct
    return (struct * len(kvs))(*[kv.struct for kv in kvs])


def layer_prefill_kv(cfg: Config, layer: PackedLayer, x: torch.Tensor, pos: torch.Tensor,
                     kv: Union[KvCache, KvCacheQ8], seq: int = 0, ds_slab: Optional[torch.Tensor] = None,
                     ds_rows: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """layer_prefill that also writes rows 0..S-1 of cache slot `seq` (bf16 or 8-bit)."""
    S = x.shape[0]
    ws = workspace(cfg, S, x.device) if ws is None else ws
    n_img = 0 if ds_rows is None else ds_rows.numel()
    fn = lib().q3vl_layer_prefill_kv_q8 if _is_q8([kv]) else lib().q3vl_layer_prefill_kv
    _check(fn(ctypes.byref(cfg), ctypes.byref(layer.views), _ptr(x), S, _ptr(pos), _ptr(ds_slab),
              _ptr(ds_rows), n_img, ctypes.byref(kv.struct), seq, _ptr(ws), ws.numel(),
              _stream(stream)))
    return x


def stack_prefill_kv(cfg: Config, layers: Sequence[PackedLayer], x: torch.Tensor,
                     pos: torch.Tensor, kvs: Sequence[Union[KvCache, KvCacheQ8]], seq: int = 0,
                     final_norm: Optional[torch.Tensor] = None,
                     ds_slabs: Sequence[torch.Tensor] = (), ds_rows: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """stack_prefill that also writes each layer's rows 0..S-1 of cache slot `seq` (caches all
    bf16 or all 8-bit)."""
    S = x.shape[0]
    ws = workspace(cfg, S, x.device) if ws is None else ws
    arr = (Layer * len(layers))(*[l.views for l in layers])
    slabs = (ctypes.c_void_p * max(1, len(ds_slabs)))(*[s.data_ptr() for s in ds_slabs])
    n_img = 0 if ds_rows is None else ds_rows.numel()
    fn = lib().q3vl_stack_prefill_kv_q8 if _is_q8(kvs) else lib().q3vl_stack_prefill_kv
    _check(fn(ctypes.byref(cfg), len(layers), arr, _ptr(final_norm), _ptr(x), S, _ptr(pos),
              slabs if ds_slabs else None, len(ds_slabs), _ptr(ds_rows), n_img, _kv_array(kvs),
              seq, _ptr(ws), ws.numel(), _stream(stream)))
    return x


def decode_workspace_bytes(cfg: Config, B: int, cap: int, dtype="bf16") -> int:
    """dtype: the caches' ("bf16" or "fp8")."""
    fn = lib().q3vl_decode_workspace_bytes if dtype == "bf16" else \
        lib().q3vl_decode_q8_workspace_bytes
    return int(fn(ctypes.byref(cfg), B, cap))


def decode_workspace(cfg: Config, B: int, cap: int, device="cuda", dtype="bf16") -> torch.Tensor:
    n = decode_workspace_bytes(cfg, B, cap, dtype)
    if n == 0:
        _check(_abi.EINVAL)
    return torch.empty(n, dtype=torch.uint8, device=device)


def layer_decode(cfg: Config, layer: PackedLayer, x: torch.Tensor, pos: torch.Tensor,
                 kv: Union[KvCache, KvCacheQ8], seq: torch.Tensor, lens: torch.Tensor,
                 ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One new token per sequence (x [B, H] in place): token b's K/V go to row lens[b] of
    slot seq[b], and it attends to rows 0..lens[b] of that slot."""
    B = x.shape[0]
    q8 = _is_q8([kv])
    if ws is None:
        ws = decode_workspace(cfg, B, kv.cap, x.device, "fp8" if q8 else "bf16")
    fn = lib().q3vl_layer_decode_q8 if q8 else lib().q3vl_layer_decode
    _check(fn(ctypes.byref(cfg), ctypes.byref(layer.views), _ptr(x), B, _ptr(pos),
              ctypes.byref(kv.struct), _ptr(seq), _ptr(lens), _ptr(ws), ws.numel(),
              _stream(stream)))
    return x


def stack_decode(cfg: Config, layers: Sequence[PackedLayer], x: torch.Tensor, pos: torch.Tensor,
                 kvs: Sequence[Union[KvCache, KvCacheQ8]], seq: torch.Tensor, lens: torch.Tensor,
                 final_norm: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """layer_decode through every layer, then the optional final norm; x in place."""
    B = x.shape[0]
    cap = max(kv.cap for kv in kvs)
    q8 = _is_q8(kvs)
    if ws is None:
        ws = decode_workspace(cfg, B, cap, x.device, "fp8" if q8 else "bf16")
    arr = (Layer * len(layers))(*[l.views for l in layers])
    fn = lib().q3vl_stack_decode_q8 if q8 else lib().q3vl_stack_decode
    _check(fn(ctypes.byref(cfg), len(layers), arr, _ptr(final_norm), _ptr(x), B, _ptr(pos),
              _kv_array(kvs), _ptr(seq), _ptr(lens), _ptr(ws), ws.numel(), _stream(stream)))
    return x


def decode_advance(pos: torch.Tensor, lens: torch.Tensor, stream=None) -> None:
    """lens += 1 and every position axis += 1 (the next text token), on the device."""
    _check(lib().q3vl_decode_advance(lens.numel(), _ptr(pos), _ptr(lens), _stream(stream)))


# ---------------------------------------------------------------------------
# Embedding gather (+ soft-token splice) and LM head
# ---------------------------------------------------------------------------
def embed(cfg: Config, table: torch.Tensor, tokens: torch.Tensor,
          soft: Optional[torch.Tensor] = None, soft_rows: Optional[torch.Tensor] = None,
          x: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x[p] = table[tokens[p]], then x[soft_rows[k]] = soft[k]; returns x [S, H]."""
    S = tokens.numel()
    x = torch.empty((S, cfg.hidden), dtype=table.dtype, device=table.device) if x is None else x
    n_soft = 0 if soft_rows is None else soft_rows.numel()
    ws = torch.empty(max(1, 4 * S), dtype=torch.uint8, device=table.device) if n_soft else None
    _check(lib().q3vl_embed(ctypes.byref(cfg), _ptr(table), table.shape[0], _ptr(tokens), S,
                           _ptr(soft), _ptr(soft_rows), n_soft, _ptr(x), _ptr(ws),
                           0 if ws is None else ws.numel(), _stream(stream)))
    return x


def lm_head(cfg: Config, x_rows: torch.Tensor, final_norm: Optional[torch.Tensor],
            weight: Union[torch.Tensor, "LinearQ8"], logits: Optional[torch.Tensor] = None,
            ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """logits [B, vocab] fp32 = RMSNorm(x_rows, final_norm) weight^T (weight: [vocab, H], bf16
    or its 8-bit form, with which the normalised rows are quantised too)."""
    if isinstance(weight, LinearQ8):
        return _lm_head_q8(cfg, x_rows, final_norm, weight, logits, ws, stream)
    B, vocab = x_rows.shape[0], weight.shape[0]
    if logits is None:
        logits = torch.empty((B, vocab), dtype=torch.float32, device=x_rows.device)
    if ws is None:
        n = int(lib().q3vl_lm_head_workspace_bytes(ctypes.byref(cfg), B))
        if n == 0:
            _check(_abi.EINVAL)
        ws = torch.empty(n, dtype=torch.uint8, device=x_rows.device)
    _check(lib().q3vl_lm_head(ctypes.byref(cfg), _ptr(x_rows), B, _ptr(final_norm), _ptr(weight),
                             vocab, _ptr(logits), _ptr(ws), ws.numel(), _stream(stream)))
    return logits


# ---------------------------------------------------------------------------
# 8-bit serving: e4m3 rows, weights and cache with power-of-two block scales
# ---------------------------------------------------------------------------
_ROW_TYPES = (torch.bfloat16, torch.float32)


def _arg(t: torch.Tensor, name: str, dtypes, shape=None, device=None) -> None:
    """Raises unless t is a contiguous tensor of one of `dtypes` (and the shape and device)."""
    if not isinstance(t, torch.Tensor):
        raise Q3VLError(_abi.EINVAL, f"{name} must be a tensor")
    if t.dtype not in dtypes:
        raise Q3VLError(_abi.EINVAL, f"{name} must be {' or '.join(map(str, dtypes))}, not {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise Q3VLError(_abi.EINVAL, f"{name} must be {tuple(shape)}, not {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise Q3VLError(_abi.EINVAL, f"{name} is on {t.device}, not {device}")
    if not t.is_contiguous():
        raise Q3VLError(_abi.EINVAL, f"{name} must be contiguous")


def _is(t, dtype, shape, index: int) -> bool:
    """Whether _arg would accept t on CUDA device `index`, at a fraction of its cost."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and
            t.get_device() == index and t.is_contiguous())


def _run(t: torch.Tensor, index: int, stream, call, *args):
    """call(*args, stream handle) with t's device current (`index`; the library works on the
    current one) and, where a stream is given, with it current, so that what `call` allocates
    belongs to it."""
    if stream is None and index >= 0 and index == _device():
        return call(*args, _raw_stream(index))
    with _on(t, stream) as st:
        return call(*args, st)


class _on:
    """The device and stream guards of _run; gives the stream to launch on."""

    def __init__(self, t: torch.Tensor, stream=None):
        if t.device.type != "cuda":
            raise Q3VLError(_abi.EINVAL, f"tensors must be on a CUDA device, not {t.device}")
        if stream is not None and stream.device != t.device:
            raise Q3VLError(_abi.EINVAL, f"the stream is on {stream.device}, tensors on {t.device}")
        self.device, self.stream, self.guards = t.device, stream, []

    def __enter__(self):
        if self.device.index != torch.cuda.current_device():
            self.guards.append(torch.cuda.device(self.device))
        if self.stream is not None:
            self.guards.append(torch.cuda.stream(self.stream))
        for guard in self.guards:
            guard.__enter__()
        return _stream(self.stream)

    def __exit__(self, *exc):
        for guard in reversed(self.guards):
            guard.__exit__(*exc)


class LinearQ8:
    """An 8-bit weight: e4m3 [N, K] with E8M0 scales [ceil(N/128), ceil(K/128)]."""

    def __init__(self, weight: torch.Tensor, scales: torch.Tensor):
        _arg(weight, "weight", (torch.float8_e4m3fn,))
        if weight.dim() != 2:
            raise Q3VLError(_abi.EINVAL, f"weight must be [N, K], not {tuple(weight.shape)}")
        N, K = weight.shape
        _arg(scales, "scales", (torch.float8_e8m0fnu,), (-(-N // Q8_BLOCK), -(-K // Q8_BLOCK)),
             weight.device)
        self.weight, self.scales = weight, scales
        self._index = weight.get_device()

    @property
    def shape(self) -> Tuple[int, int]:
        return tuple(self.weight.shape)


def quantize_weight_q8(w: torch.Tensor, stream=None) -> LinearQ8:
    """The 8-bit form of a weight [N, K] (bf16 or fp32), one scale per 128 x 128 block."""
    _arg(w, "w", _ROW_TYPES)
    if w.dim() != 2:
        raise Q3VLError(_abi.EINVAL, f"w must be [N, K], not {tuple(w.shape)}")
    N, K = w.shape
    cfg = config(128, 1, 1, 128, "bf16" if w.dtype == torch.bfloat16 else "fp32")

    def call(st):
        wq = torch.empty((N, K), dtype=torch.float8_e4m3fn, device=w.device)
        ws = torch.empty((-(-N // Q8_BLOCK), -(-K // Q8_BLOCK)), dtype=torch.float8_e8m0fnu,
                         device=w.device)
        _check(lib().q3vl_quantize_weight_q8(ctypes.byref(cfg), _ptr(w), N, K, _ptr(wq), _ptr(ws),
                                             st))
        return LinearQ8(wq, ws)
    return _run(w, w.get_device(), stream, call)


def add_rms_norm_q8(cfg: Config, x: torch.Tensor, gain: Optional[torch.Tensor],
                    delta: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(h, q, scales): h = x + delta (x itself without a delta), and the 8-bit form of
    RMSNorm(h) * gain: e4m3 [S, H] with E8M0 scales [S, ceil(H/128)].

    gain None quantises h without a norm; a bf16 gain of 2^64 or more is a device error. h: where
    to write the sum (x for in place); a new tensor by default.
    """
    dt = torch_dtype(cfg)
    if not (isinstance(x, torch.Tensor) and x.dtype is dt and x.is_contiguous()):
        _arg(x, "x", (dt,))
    shape, index = x.shape, x.get_device()
    if len(shape) != 2 or shape[1] != cfg.hidden:
        raise Q3VLError(_abi.EINVAL, f"x must be [S, {cfg.hidden}], not {tuple(x.shape)}")
    if gain is not None and not _is(gain, dt, shape[1:], index):
        _arg(gain, "gain", (dt,), shape[1:], x.device)
    if delta is None:
        if h is not None and h is not x:
            raise Q3VLError(_abi.EINVAL, "without a delta, h is x")
        h = x
    else:
        if not _is(delta, dt, shape, index):
            _arg(delta, "delta", (dt,), shape, x.device)
        if h is not None and not _is(h, dt, shape, index):
            _arg(h, "h", (dt,), shape, x.device)
    return _run(x, index, stream, _add_rms_norm_q8, cfg, x, gain, delta, h)


def _add_rms_norm_q8(cfg, x, gain, delta, h, st):
    S, H = x.shape
    if h is None:
        h = torch.empty_like(x)
    q = torch.empty_like(x, dtype=torch.float8_e4m3fn)
    sc = x.new_empty(S, -(-H // Q8_BLOCK), dtype=torch.float8_e8m0fnu)
    rc = lib().q3vl_add_rms_norm_q8(
        ctypes.byref(cfg), x.data_ptr(), None if delta is None else delta.data_ptr(), S,
        None if gain is None else gain.data_ptr(), h.data_ptr(), q.data_ptr(), sc.data_ptr(), st)
    if rc:
        _check(rc)
    return h, q, sc


def linear_q8(xq: torch.Tensor, scales: torch.Tensor, lin: LinearQ8,
              resid: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """[M, N] = x W^T (+ resid) of 8-bit rows (as add_rms_norm_q8 gives them) and an 8-bit
    weight, summed in fp32 and rounded once to out_dtype (bfloat16 or float32)."""
    if not (isinstance(xq, torch.Tensor) and xq.dtype is torch.float8_e4m3fn and
            xq.is_contiguous()):
        _arg(xq, "xq", (torch.float8_e4m3fn,))
    if not isinstance(lin, LinearQ8):
        raise Q3VLError(_abi.EINVAL, "lin must be a LinearQ8")
    N, K = lin.weight.shape
    shape, index = xq.shape, xq.get_device()
    if len(shape) != 2 or shape[1] != K:
        raise Q3VLError(_abi.EINVAL, f"xq must be [M, {K}], not {tuple(xq.shape)}")
    M = shape[0]
    if not _is(scales, torch.float8_e8m0fnu, (M, -(-K // Q8_BLOCK)), index):
        _arg(scales, "scales", (torch.float8_e8m0fnu,), (M, -(-K // Q8_BLOCK)), xq.device)
    if lin._index != index:
        raise Q3VLError(_abi.EINVAL, f"the weight is on {lin.weight.device}, xq on {xq.device}")
    if out_dtype not in _ROW_TYPES:
        raise Q3VLError(_abi.EUNSUPPORTED, f"out_dtype must be bfloat16 or float32, not {out_dtype}")
    if resid is not None and not _is(resid, out_dtype, (M, N), index):
        _arg(resid, "resid", (out_dtype,), (M, N), xq.device)
    if out is not None and not _is(out, out_dtype, (M, N), index):
        _arg(out, "out", (out_dtype,), (M, N), xq.device)
    return _run(xq, index, stream, _linear_q8, xq, scales, lin, resid, out_dtype, out, M, N, K)


def _linear_q8(xq, scales, lin, resid, out_dtype, out, M, N, K, st):
    if out is None:
        out = xq.new_empty(M, N, dtype=out_dtype)
    rc = lib().q3vl_linear_q8(
        xq.data_ptr(), scales.data_ptr(), M, lin.weight.data_ptr(), lin.scales.data_ptr(), N, K,
        None if resid is None else resid.data_ptr(), out.data_ptr(),
        _abi.DTYPE_BF16 if out_dtype is torch.bfloat16 else _abi.DTYPE_FP32, st)
    if rc:
        _check(rc)
    return out


def _lm_head_q8(cfg, x_rows, final_norm, lin, logits, ws, stream):
    _arg(x_rows, "x_rows", (torch.bfloat16,))
    vocab, K = lin.shape
    if x_rows.dim() != 2 or x_rows.shape[1] != cfg.hidden or K != cfg.hidden:
        raise Q3VLError(_abi.EINVAL, f"x_rows and weight must have {cfg.hidden} columns")
    B = x_rows.shape[0]
    if final_norm is not None:
        _arg(final_norm, "final_norm", (torch.bfloat16,), (cfg.hidden,), x_rows.device)
    if lin.weight.device != x_rows.device:
        raise Q3VLError(_abi.EINVAL, f"the weight is on {lin.weight.device}, x_rows on {x_rows.device}")
    if logits is not None:
        _arg(logits, "logits", (torch.float32,), (B, vocab), x_rows.device)
    if ws is not None:
        _arg(ws, "ws", (torch.uint8,), None, x_rows.device)

    def call(logits, ws, st):
        if logits is None:
            logits = torch.empty((B, vocab), dtype=torch.float32, device=x_rows.device)
        if ws is None:
            n = int(lib().q3vl_lm_head_q8_workspace_bytes(ctypes.byref(cfg), B))
            if n == 0:
                _check(_abi.EINVAL)
            ws = torch.empty(n, dtype=torch.uint8, device=x_rows.device)
        _check(lib().q3vl_lm_head_q8(ctypes.byref(cfg), _ptr(x_rows), B, _ptr(final_norm),
                                     _ptr(lin.weight), _ptr(lin.scales), vocab, _ptr(logits),
                                     _ptr(ws), ws.numel(), st))
        return logits
    return _run(x_rows, x_rows.get_device(), stream, call, logits, ws)


def _ints(t: torch.Tensor, name: str, n: int, kv: KvCacheQ8) -> None:
    if not _is(t, torch.int32, (n,), kv._index):
        _arg(t, name, (torch.int32,), (n,), kv.k.device)


def kv_store_q8(cfg: Config, k: torch.Tensor, v: torch.Tensor, kv: KvCacheQ8, seq: torch.Tensor,
                lens: torch.Tensor, starts: Optional[torch.Tensor] = None, stream=None) -> None:
    """Appends rows to sequences of an 8-bit cache: rows starts[b]..starts[b+1]-1 of k and v go to
    rows lens[b].. of slot seq[b] (without starts, row b alone).

    k, v: bf16 [T, nkv*128] with contiguous rows and one row stride, such as the k and v column
    ranges of a QKV buffer. seq (distinct slots) and lens: int32 [B]; starts: int32 [B+1]. lens
    is not advanced.
    """
    if not isinstance(kv, KvCacheQ8):
        raise Q3VLError(_abi.EINVAL, "kv must be a KvCacheQ8")
    if not (isinstance(k, torch.Tensor) and isinstance(v, torch.Tensor) and
            isinstance(seq, torch.Tensor)):
        raise Q3VLError(_abi.EINVAL, "k, v and seq must be tensors")
    dkv, index = cfg.n_kv_heads * cfg.head_dim, kv._index
    shape, strides = k.shape, k.stride()
    T, B = shape[0] if shape else 0, seq.numel()
    # rows of dkv elements, one shape, type, stride and device
    if not (k.dtype is torch.bfloat16 and v.dtype is torch.bfloat16 and
            len(shape) == 2 and shape[1] == dkv and v.shape == shape and strides[1] == 1 and
            strides[0] >= dkv and v.stride() == strides and k.get_device() == index and
            v.get_device() == index):
        _kv_rows(k, v, dkv, kv)
    if kv._width != dkv:
        raise Q3VLError(_abi.EINVAL, f"the cache has rows of {kv._width}, the config {dkv}")
    _ints(seq, "seq", B, kv)
    _ints(lens, "lens", B, kv)
    if starts is not None:
        _ints(starts, "starts", B + 1, kv)
    ld = strides[0] if T > 1 else dkv
    _run(k, index, stream, _kv_store_q8, cfg, k, v, ld, T, starts, B, kv, seq, lens)


def _kv_rows(k, v, dkv, kv) -> None:
    """What kv_store_q8 asks of k and v, one by one (a single row may have any stride)."""
    for t, name in ((k, "k"), (v, "v")):
        if t.dtype != torch.bfloat16 or t.dim() != 2 or t.shape[1] != dkv:
            raise Q3VLError(_abi.EINVAL, f"{name} must be bfloat16 [T, {dkv}], not "
                                         f"{t.dtype} {tuple(t.shape)}")
        if t.shape[0] > 0 and (t.stride(1) != 1 or (t.shape[0] > 1 and t.stride(0) < dkv)):
            raise Q3VLError(_abi.EINVAL, f"{name} must have contiguous rows that do not overlap")
        if t.device != kv.k.device:
            raise Q3VLError(_abi.EINVAL, f"{name} is on {t.device}, the cache on {kv.k.device}")
    if v.shape != k.shape or (k.shape[0] > 1 and v.stride(0) != k.stride(0)):
        raise Q3VLError(_abi.EINVAL, "k and v must have one shape and row stride")


def _kv_store_q8(cfg, k, v, ld, T, starts, B, kv, seq, lens, st):
    rc = lib().q3vl_kv_store_q8(ctypes.byref(cfg), k.data_ptr(), v.data_ptr(), ld, T,
                                None if starts is None else starts.data_ptr(), B,
                                ctypes.byref(kv.struct), seq.data_ptr(), lens.data_ptr(), st)
    if rc:
        _check(rc)


def attention_q8_workspace(cfg: Config, B: int, cap: int, device="cuda") -> torch.Tensor:
    n = int(lib().q3vl_attention_q8_workspace_bytes(ctypes.byref(cfg), B, cap))
    if n == 0:
        _check(_abi.EINVAL)
    return torch.empty(n, dtype=torch.uint8, device=device)


def attention_q8(cfg: Config, q: torch.Tensor, kv: KvCacheQ8, seq: torch.Tensor,
                 lens: torch.Tensor, o: Optional[torch.Tensor] = None,
                 ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """o [B, nh*128] bf16: the attention of query row b (q [B, nh*128] bf16) over rows
    0..lens[b]-1 of slot seq[b] of an 8-bit cache; a length of 0 gives a zero row."""
    if not isinstance(kv, KvCacheQ8):
        raise Q3VLError(_abi.EINVAL, "kv must be a KvCacheQ8")
    dq, dkv = cfg.n_heads * cfg.head_dim, cfg.n_kv_heads * cfg.head_dim
    if not (isinstance(q, torch.Tensor) and q.dtype is torch.bfloat16 and q.is_contiguous()):
        _arg(q, "q", (torch.bfloat16,))
    shape, index = q.shape, q.get_device()
    if len(shape) != 2 or shape[1] != dq:
        raise Q3VLError(_abi.EINVAL, f"q must be [B, {dq}], not {tuple(q.shape)}")
    if kv._width != dkv:
        raise Q3VLError(_abi.EINVAL, f"the cache has rows of {kv._width}, the config {dkv}")
    if kv._index != index:
        raise Q3VLError(_abi.EINVAL, f"the cache is on {kv.k.device}, q on {q.device}")
    B = shape[0]
    _ints(seq, "seq", B, kv)
    _ints(lens, "lens", B, kv)
    if o is not None and not _is(o, torch.bfloat16, shape, index):
        _arg(o, "o", (torch.bfloat16,), (B, dq), q.device)
    if ws is not None:
        _arg(ws, "ws", (torch.uint8,), None, q.device)
    return _run(q, index, stream, _attention_q8, cfg, q, B, kv, seq, lens, o, ws)


def _attention_q8(cfg, q, B, kv, seq, lens, o, ws, st):
    if o is None:
        o = torch.empty_like(q)
    if ws is None:
        ws = attention_q8_workspace(cfg, B, kv.cap, q.device)
    rc = lib().q3vl_attention_q8(ctypes.byref(cfg), q.data_ptr(), B, ctypes.byref(kv.struct),
                                 seq.data_ptr(), lens.data_ptr(), o.data_ptr(), ws.data_ptr(),
                                 ws.numel(), st)
    if rc:
        _check(rc)
    return o


# ---------------------------------------------------------------------------
# Step-level calls
# ---------------------------------------------------------------------------
def rope_table(cfg: Config, pos: torch.Tensor, stream=None) -> torch.Tensor:
    S = pos.shape[1]
    cs = torch.empty((S, 64, 2), dtype=torch.float32, device=pos.device)
    _check(lib().q3vl_rope_table(ctypes.byref(cfg), _ptr(pos), S, _ptr(cs), _stream(stream)))
    return cs


def rms_rowstat(cfg: Config, x: torch.Tensor, stream=None) -> torch.Tensor:
    S, width = x.shape
    inv = torch.empty(S, dtype=torch.float32, device=x.device)
    _check(lib().q3vl_rms_rowstat(ctypes.byref(cfg), _ptr(x), S, width, _ptr(inv),
                                 _stream(stream)))
    return inv


def _qkv_dim(cfg: Config) -> int:
    return (cfg.n_heads + 2 * cfg.n_kv_heads) * cfg.head_dim


def qkv_proj(cfg, layer: PackedLayer, x, inv_rms, cos_sin, ws=None, stream=None) -> torch.Tensor:
    S = x.shape[0]
    ws = workspace(cfg, S, x.device) if ws is None else ws
    qkv = torch.empty((S, _qkv_dim(cfg)), dtype=x.dtype, device=x.device)
    _check(lib().q3vl_qkv_proj(ctypes.byref(cfg), ctypes.byref(layer.views), _ptr(x), S,
                              _ptr(inv_rms), _ptr(cos_sin), _ptr(qkv), _ptr(ws), ws.numel(),
                              _stream(stream)))
    return qkv


def attention(cfg, qkv, stream=None) -> torch.Tensor:
    S = qkv.shape[0]
    o = torch.empty((S, cfg.n_heads * cfg.head_dim), dtype=qkv.dtype, device=qkv.device)
    _check(lib().q3vl_attention(ctypes.byref(cfg), _ptr(qkv), S, _ptr(o), _stream(stream)))
    return o


def o_proj(cfg, layer: PackedLayer, o, x, ws=None, stream=None) -> torch.Tensor:
    S = o.shape[0]
    ws = workspace(cfg, S, o.device) if ws is None else ws
    h = torch.empty((S, cfg.hidden), dtype=o.dtype, device=o.device)
    _check(lib().q3vl_o_proj(ctypes.byref(cfg), ctypes.byref(layer.views), _ptr(o), _ptr(x), S,
                            _ptr(h), _ptr(ws), ws.numel(), _stream(stream)))
    return h


def gate_up(cfg, layer: PackedLayer, h, inv_rms2, ws=None, stream=None) -> torch.Tensor:
    S = h.shape[0]
    ws = workspace(cfg, S, h.device) if ws is None else ws
    act = torch.empty((S, cfg.intermediate), dtype=h.dtype, device=h.device)
    _check(lib().q3vl_gate_up(ctypes.byref(cfg), ctypes.byref(layer.views), _ptr(h), S,
                             _ptr(inv_rms2), _ptr(act), _ptr(ws), ws.numel(), _stream(stream)))
    return act


def down(cfg, layer: PackedLayer, act, h, ds_slab=None, ds_map=None, ws=None,
         stream=None) -> torch.Tensor:
    S = act.shape[0]
    ws = workspace(cfg, S, act.device) if ws is None else ws
    out = torch.empty((S, cfg.hidden), dtype=act.dtype, device=act.device)
    _check(lib().q3vl_down(ctypes.byref(cfg), ctypes.byref(layer.views), _ptr(act), _ptr(h), S,
                          _ptr(ds_slab), _ptr(ds_map), _ptr(out), _ptr(ws), ws.numel(),
                          _stream(stream)))
    return out


def deepstack_map(ds_rows: torch.Tensor, S: int, stream=None) -> torch.Tensor:
    m = torch.empty(S, dtype=torch.int32, device=ds_rows.device)
    _check(lib().q3vl_deepstack_map(_ptr(ds_rows), ds_rows.numel(), S, _ptr(m), _stream(stream)))
    return m


def final_norm(cfg, x, gain, stream=None) -> torch.Tensor:
    _check(lib().q3vl_final_norm(ctypes.byref(cfg), _ptr(x), x.shape[0], _ptr(gain),
                                _stream(stream)))
    return x


def device_status(stream=None):
    """Synchronises and returns (code, where) of the device error record, clearing it."""
    code, where = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(lib().q3vl_device_status(_stream(stream), ctypes.byref(code), ctypes.byref(where)))
    return code.value, where.value


def check_device(stream=None) -> None:
    code, where = device_status(stream)
    if code != _abi.OK:
        raise Q3VLError(code, f"device-side error at location {where}")


def selftest_wait_timeout(timeout_us: int, stream=None) -> None:
    _check(lib().q3vl_selftest_wait_timeout(timeout_us, _stream(stream)))


def set_stage_events(events) -> None:
    """Records the 9 stage-boundary events in each following layer_prefill call
    (torch.cuda.Event(enable_timing=True) objects); None stops recording."""
    if events is None:
        _check(lib().q3vl_set_stage_events(None, 0))
        return
    for e in events:
        if e.cuda_event == 0:
            e.record()  # torch creates the CUDA event on first record
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(lib().q3vl_set_stage_events(arr, len(events)))


def launch_count() -> int:
    """Kernels enqueued by the library so far in this process."""
    return int(lib().q3vl_launch_count())
