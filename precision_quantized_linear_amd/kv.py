"""Cache of keys and values: rotary positions, slots of a batch's new tokens, quantizing keys and
values as they are written, reading them back, and the attention over the pages.

Argument marshalling only, as in the package's other calls: every step runs in the HIP kernels of
``libpql.so`` (include/pql.h, "cache of keys and values").  For inference: no call records a
gradient.

    cache = kv_cache(n_pages, 64, 8, 128)                            # per layer, once
    turn = rope_freqs(128, base=10000.0, device="cuda")              # once
    slots, positions = kv_slots(starts, lens, pages, 64, T)          # once a step
    kv_append(k, v, cache, slots, turn, positions)                   # per layer
    y = kv_attention(rope(q, positions, turn), cache, starts, lens, pages)
"""
from __future__ import annotations

import ctypes
import functools
import math
import sys
from dataclasses import dataclass

import torch

from . import _call, _check, _check_vector, _on_device, _ptr, lib

KV_SCHEMES = {"bf16": 0, "fp8_tensor": 1, "fp8_row": 2}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
KV_HEAD_DIMS = (64, 128, 192, 256)


# ---------------------------------------------------------------- rotary positions
@dataclass
class Rope:
    """A table of rotary frequencies: ``freqs`` (device float64 [rotary / 2], radians per position),
    ``scale`` (on the turned values), ``layout``: pairs (i, i + rotary / 2) "half", or (2 i, 2 i + 1)
    "interleaved"."""
    freqs: torch.Tensor
    scale: float = 1.0
    layout: str = "half"


def rope_freqs(dim: int, base: float = 10000.0, *, layout: str = "half", scaling: dict | None = None,
               device=None) -> Rope:
    """The table for ``dim`` turned values of a head: base^(-2 i / dim), stretched for contexts
    longer than the model was trained on by ``scaling`` (a dict; s = its "factor"):

    * {"type": "linear", "factor"}: every frequency / s.
    * {"type": "ntk", "factor"}: the base times s^(dim / (dim - 2)).
    * {"type": "yarn", "factor", "original", "fast" = 32, "slow" = 1, "attention" = 0.1 ln s + 1}: pairs that
      turn more than ``fast`` times over ``original`` positions keep their frequency, those that turn
      less than ``slow`` times get it / s, a straight ramp over the pair's index lies between; the turned
      values are multiplied by ``attention``.
    * {"type": "bands", "factor", "original", "fast" = 4, "slow" = 1}: the same two ends, and between them
      the ramp is straight in the number of turns."""
    if not isinstance(dim, int) or dim < 16 or dim % 16:
        raise ValueError(f"dim must be a multiple of 16 (got {dim!r})")
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"unknown layout {layout!r}; supported: {sorted(ROPE_LAYOUTS)}")
    if not (base > 1.0 and math.isfinite(base)):
        raise ValueError(f"base must be a finite number above 1 (got {base!r})")
    scaling = dict(scaling or {"type": "none"})
    kind, known = scaling.pop("type", None), {"none": (), "linear": ("factor",), "ntk": ("factor",),
                                              "yarn": ("factor", "original", "fast", "slow", "attention"),
                                              "bands": ("factor", "original", "fast", "slow")}
    if kind not in known:
        raise ValueError(f"unknown scaling {kind!r}; supported: {sorted(known)}")
    if set(scaling) - set(known[kind]):
        raise ValueError(f"{kind} scaling does not take {sorted(set(scaling) - set(known[kind]))}")
    missing = [k for k in known[kind] if k in ("factor", "original") and k not in scaling]
    if missing:
        raise ValueError(f"{kind} scaling needs {missing}")
    s = float(scaling.get("factor", 1.0))
    if not (s >= 1.0 and math.isfinite(s)):
        raise ValueError(f"factor must be a finite number from 1 on (got {s!r})")
    if kind == "ntk":
        if math.log(base) + math.log(s) * dim / (dim - 2) >= math.log(sys.float_info.max):
            raise ValueError(f"ntk scaling needs a factor whose base is finite (got {s!r})")
        base *= s ** (dim / (dim - 2))
    pairs = torch.arange(dim // 2, dtype=torch.float64)
    f = base ** (-2.0 * pairs / dim)
    scale = 1.0
    if kind == "linear":
        f = f / s
    elif kind in ("yarn", "bands"):
        span = float(scaling["original"])
        fast, slow = float(scaling.get("fast", 32.0 if kind == "yarn" else 4.0)), float(scaling.get("slow", 1.0))
        if not (span > 0 and fast > slow > 0):
            raise ValueError(f"{kind} scaling needs original > 0 and fast > slow > 0")
        if kind == "yarn":
            if not (math.isfinite(span) and math.isfinite(fast)):
                raise ValueError("yarn scaling needs finite original and fast")

            def pair_of(turns):   # the (real) index whose frequency turns so often over `original` positions
                return dim * math.log(span / (2 * math.pi * turns)) / (2 * math.log(base))
            lo = max(math.floor(pair_of(fast)), 0)
            hi = min(math.ceil(pair_of(slow)), dim - 1)
            keep = 1.0 - ((pairs - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
            scale = float(scaling.get("attention", 0.1 * math.log(s) + 1.0))
            if not math.isfinite(ctypes.c_float(scale).value):
                raise ValueError(f"yarn scaling needs an attention that is finite in float32 (got {scale!r})")
        else:
            keep = ((span * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f * keep + f / s * (1.0 - keep)
    return Rope(f if device is None else f.to(device), scale, layout)


def _heads(t, name: str, device=None):
    """The sizes and strides of a bf16 [n, H, D] operand on ``device``, its D values contiguous."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be a bfloat16 tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head size], not {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the operands on {device}")
    (n, H, D), (st, sh, unit) = t.shape, t.stride()
    if unit != 1 and D > 1:
        raise ValueError(f"{name} must have unit stride along the head")
    # the stride of an axis of one has no meaning; torch may give any
    if H == 1:
        sh = D
    if n <= 1:
        st = sh * H
    return n, H, D, st, sh


def _check_rope(table, D: int, device) -> int:
    if not isinstance(table, Rope):
        raise ValueError("the rotary table must be a Rope")
    if table.layout not in ROPE_LAYOUTS:
        raise ValueError(f"unknown layout {table.layout!r}; supported: {sorted(ROPE_LAYOUTS)}")
    f = table.freqs
    if not isinstance(f, torch.Tensor) or f.dtype is not torch.float64 or f.dim() != 1 or not f.is_contiguous():
        raise ValueError("freqs must be a contiguous 1-D float64 tensor")
    if f.device != device:
        raise ValueError(f"freqs are on {f.device}, the operands on {device}")
    if 2 * f.numel() > D:
        raise ValueError(f"{f.numel()} pairs do not fit a head of {D}")
    return 2 * f.numel()


def rope(x: torch.Tensor, positions: torch.Tensor, table: Rope, out: torch.Tensor | None = None) -> torch.Tensor:
    """Turn the heads of bf16 x [T, H, D] by int32 ``positions`` [T]; values behind the table's stay as
    they are.  x may be a view with any strides that are multiples of 8 (heads of a wider projection);
    ``out`` may be x itself."""
    T, H, D, st, sh = _heads(x, "x")
    device = x.device
    rotary = _check_rope(table, D, device)
    _check_vector(positions, "positions", torch.int32, T, device)
    if out is None:
        out, ot, oh = torch.empty((T, H, D), dtype=torch.bfloat16, device=device), H * D, D
    else:
        n, h, d, ot, oh = _heads(out, "out", device)
        if (n, h, d) != (T, H, D):
            raise ValueError(f"out must be {(T, H, D)}, not {(n, h, d)}")
    _on_device(device)
    _call(lib().pql_rope, "rope", device, ROPE_LAYOUTS[table.layout], x.data_ptr(), T, H, D, st, sh, positions.data_ptr(),
          table.freqs.data_ptr(), rotary, table.scale, out.data_ptr(), ot, oh)
    return out


# ---------------------------------------------------------------- the cache
@dataclass
class KVCache:
    """Pages of keys and values, [n_pages, n_kv_heads, page_size, head_dim] each: bfloat16 under "bf16",
    e4m3 codes (uint8) under "fp8_tensor" and "fp8_row", with float32 scales ([1], or
    [n_pages, n_kv_heads, page_size])."""
    scheme: str
    n_pages: int
    page_size: int
    n_kv_heads: int
    head_dim: int
    k: torch.Tensor
    v: torch.Tensor
    k_scales: torch.Tensor | None = None
    v_scales: torch.Tensor | None = None

    @property
    def device(self):
        return self.k.device


def _kv_scheme(scheme: str) -> int:
    if scheme not in KV_SCHEMES:
        raise ValueError(f"unknown cache scheme {scheme!r}; supported: {sorted(KV_SCHEMES)}")
    return KV_SCHEMES[scheme]


def kv_sizes(scheme: str, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int):
    """(codes bytes, scales bytes) of each of a cache's two halves."""
    c, s = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().pql_kv_sizes(_kv_scheme(scheme), n_pages, page_size, n_kv_heads, head_dim, ctypes.byref(c),
                              ctypes.byref(s)), "kv_sizes")
    return c.value, s.value


def kv_cache(n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, scheme: str = "fp8_row", *,
             k_scale: float | None = None, v_scale: float | None = None, device="cuda") -> KVCache:
    """An empty cache (its memory is not initialised, and needs not be).  "fp8_tensor" takes the two
    scales it quantizes with, finite and positive in float32."""
    kv_sizes(scheme, n_pages, page_size, n_kv_heads, head_dim)   # refuses what no cache can be
    given = (k_scale, v_scale)
    if scheme == "fp8_tensor":
        if any(s is None or not 0.0 < ctypes.c_float(float(s)).value < math.inf for s in given):
            raise ValueError("fp8_tensor needs k_scale and v_scale, finite and positive in float32")
    elif given != (None, None):
        raise ValueError(f"{scheme} takes no k_scale and v_scale")
    shape = (n_pages, n_kv_heads, page_size, head_dim)
    kv = [torch.empty(shape, dtype=torch.bfloat16 if scheme == "bf16" else torch.uint8, device=device) for _ in "kv"]
    if scheme == "bf16":
        scales = [None, None]
    elif scheme == "fp8_tensor":
        scales = [torch.tensor([float(s)], dtype=torch.float32, device=device) for s in given]
    else:
        scales = [torch.empty(shape[:3], dtype=torch.float32, device=device) for _ in "kv"]
    return KVCache(scheme, n_pages, page_size, n_kv_heads, head_dim, *kv, *scales)


def _check_cache(c, device) -> None:
    if not isinstance(c, KVCache):
        raise ValueError("cache must be a KVCache")
    _kv_scheme(c.scheme)
    shape = (c.n_pages, c.n_kv_heads, c.page_size, c.head_dim)
    dtype = torch.bfloat16 if c.scheme == "bf16" else torch.uint8
    for t, name in ((c.k, "k"), (c.v, "v")):
        if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"cache.{name} must be a contiguous {dtype} tensor of {shape}")
        if t.device != device:
            raise ValueError(f"cache.{name} is on {t.device}, the operands on {device}")
    if c.scheme != "bf16":
        n = 1 if c.scheme == "fp8_tensor" else c.n_pages * c.n_kv_heads * c.page_size
        _check_vector(c.k_scales, "cache.k_scales", torch.float32, n, device)
        _check_vector(c.v_scales, "cache.v_scales", torch.float32, n, device)


def _cache_args(c):
    bf16 = c.scheme == "bf16"
    return (c.k.data_ptr(), c.v.data_ptr(), None if bf16 else c.k_scales.data_ptr(),
            None if bf16 else c.v_scales.data_ptr())


def _check_batch(starts, lens, pages, device):
    """(B, width, row stride) of a batch's three int32 tensors."""
    if not isinstance(lens, torch.Tensor) or lens.dim() != 1:
        raise ValueError("lens must be a 1-D int32 tensor")
    B = lens.numel()
    _check_vector(lens, "lens", torch.int32, B, device)
    _check_vector(starts, "starts", torch.int32, B + 1, device)
    if not isinstance(pages, torch.Tensor) or pages.dtype is not torch.int32 or pages.dim() != 2 or pages.shape[0] != B:
        raise ValueError(f"pages must be an int32 [{B}, pages] tensor")
    if pages.device != device:
        raise ValueError(f"pages are on {pages.device}, the operands on {device}")
    width = pages.shape[1]
    if width > 1 and pages.stride(1) != 1:
        raise ValueError("pages must have unit stride along a sequence")
    return B, width, pages.stride(0) if B > 1 else width


def kv_slots(starts: torch.Tensor, lens: torch.Tensor, pages: torch.Tensor, page_size: int, tokens: int):
    """Slots and positions (int32 [tokens] each) of a batch's new tokens, for ``kv_append`` and ``rope``:
    the i-th of the n new tokens of sequence b is at position lens[b] - n + i, in slot
    pages[b, position // page_size] * page_size + position % page_size.  Rows of no sequence get slot -1."""
    if not isinstance(lens, torch.Tensor):
        raise ValueError("lens must be a 1-D int32 tensor")
    device = lens.device
    B, width, ldp = _check_batch(starts, lens, pages, device)
    _on_device(device)
    if not isinstance(tokens, int) or not 0 <= tokens < 1 << 31:
        raise ValueError(f"tokens must be 0 .. 2^31 - 1 (got {tokens!r})")
    slots = torch.empty((tokens,), dtype=torch.int32, device=device)
    positions = torch.empty((tokens,), dtype=torch.int32, device=device)
    _call(lib().pql_kv_slots, "kv_slots", device, starts.data_ptr(), lens.data_ptr(), pages.data_ptr(), B, width, ldp,
          page_size, tokens, slots.data_ptr(), positions.data_ptr())
    return slots, positions


def kv_append(k: torch.Tensor, v: torch.Tensor, cache: KVCache, slots: torch.Tensor, table: Rope | None = None,
              positions: torch.Tensor | None = None) -> KVCache:
    """Write bf16 keys and values [T, n_kv_heads, head_dim] into the int32 ``slots`` [T] of ``cache``,
    quantized by its scheme; slots outside the cache write nothing.  With ``table`` the keys are turned
    by int32 ``positions`` [T] first, without a rounding in between."""
    T, H, D, kt, kh = _heads(k, "k")
    device = k.device
    n, h, d, vt, vh = _heads(v, "v", device)
    _check_cache(cache, device)
    if (n, h, d) != (T, H, D) or (H, D) != (cache.n_kv_heads, cache.head_dim):
        raise ValueError(f"k and v must both be [T, {cache.n_kv_heads}, {cache.head_dim}], not {tuple(k.shape)} and "
                         f"{tuple(v.shape)}")
    _check_vector(slots, "slots", torch.int32, T, device)
    if (table is None) != (positions is None):
        raise ValueError("turning the keys takes a table and positions")
    layout = rotary = 0
    scale, freqs, at = 1.0, None, None
    if table is not None and T:
        rotary = _check_rope(table, D, device)
        _check_vector(positions, "positions", torch.int32, T, device)
        layout, scale, freqs, at = ROPE_LAYOUTS[table.layout], table.scale, table.freqs.data_ptr(), positions.data_ptr()
    _on_device(device)
    kc, vc, ks, vs = _cache_args(cache)
    _call(lib().pql_kv_append, "kv_append", device, KV_SCHEMES[cache.scheme], k.data_ptr(), kt, kh, v.data_ptr(), vt, vh,
          T, slots.data_ptr(), layout, at, freqs, rotary, scale, kc, vc, ks, vs, cache.n_pages, cache.page_size, H, D)
    return cache


def kv_read(cache: KVCache, slots: torch.Tensor, out=None):
    """Keys and values of int32 ``slots`` [n] back in bf16 [n, n_kv_heads, head_dim]; a slot outside the
    cache reads as zeros.  ``out``: a pair of tensors to write to."""
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a 1-D int32 tensor")
    device, n = slots.device, slots.numel()
    _check_vector(slots, "slots", torch.int32, n, device)
    _check_cache(cache, device)
    H, D = cache.n_kv_heads, cache.head_dim
    if out is None:
        k, v = (torch.empty((n, H, D), dtype=torch.bfloat16, device=device) for _ in "kv")
        kt, kh, vt, vh = H * D, D, H * D, D
    else:
        k, v = out
        *ks, kt, kh = _heads(k, "k out", device)
        *vs, vt, vh = _heads(v, "v out", device)
        if ks != [n, H, D] or vs != [n, H, D]:
            raise ValueError(f"out must be two tensors of {(n, H, D)}")
    _on_device(device)
    _call(lib().pql_kv_read, "kv_read", device, KV_SCHEMES[cache.scheme], *_cache_args(cache), cache.n_pages,
          cache.page_size, H, D, slots.data_ptr(), n, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh)
    return k, v


# ---------------------------------------------------------------- attention
@functools.lru_cache(maxsize=4096)
def kv_attention_workspace(scheme: str, T: int, H: int, n_kv_heads: int, head_dim: int, B: int, width: int,
                           page_size: int) -> int:
    """Workspace bytes of a ``kv_attention`` call of these sizes (width: columns of its ``pages``)."""
    wsb = ctypes.c_size_t()
    _check(lib().pql_kv_attention_workspace(_kv_scheme(scheme), T, H, n_kv_heads, head_dim, B, width, page_size,
                                            ctypes.byref(wsb)), "kv_attention")
    return wsb.value


def kv_kernel_name(scheme: str, T: int, H: int, n_kv_heads: int, head_dim: int, B: int, width: int,
                   page_size: int) -> str:
    return lib().pql_kv_kernel_name(_kv_scheme(scheme), T, H, n_kv_heads, head_dim, B, width, page_size).decode()


def kv_attention(q: torch.Tensor, cache: KVCache, starts: torch.Tensor, lens: torch.Tensor, pages: torch.Tensor, *,
                 causal: bool = True, window: int = 0, scale: float | None = None, out: torch.Tensor | None = None,
                 return_lse: bool = False, workspace: torch.Tensor | None = None):
    """Attention of a batch's new tokens, bf16 q [T, H, head_dim], over the tokens in its pages; bf16
    [T, H, head_dim], and with ``return_lse`` the float32 [T, H] logarithm of each row's sum.

    Sequence b has the rows starts[b] .. starts[b + 1] - 1 of q as its last tokens, lens[b] tokens in the
    cache (these included, so ``kv_append`` comes first) and their pages in pages[b] (all int32).  A token
    at position i sees the tokens up to i (``causal``; otherwise all of its sequence) and, with
    ``window``, none before i - ``window`` + 1.  H / n_kv_heads consecutive heads share a head
    of the cache.  ``scale``: on the products, head_dim^-0.5 by default.  Rows of no sequence are left as
    they were in ``out`` (which does not overlap q), or hold anything where it is not given.
    ``workspace``: ``kv_attention_workspace`` bytes, not shared by calls that overlap in time; allocated
    where it is not given.  More: include/pql.h, pql_kv_attention."""
    T, H, D, qt, qh = _heads(q, "q")
    device = q.device
    _check_cache(cache, device)
    if D != cache.head_dim:
        raise ValueError(f"q has heads of {D}, the cache of {cache.head_dim}")
    B, width, ldp = _check_batch(starts, lens, pages, device)
    _on_device(device)
    wsb = kv_attention_workspace(cache.scheme, T, H, cache.n_kv_heads, D, B, width, cache.page_size)
    if workspace is None:
        if wsb:
            workspace = torch.empty(wsb, dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on q's device")
    if out is None:
        out, ot, oh = torch.empty((T, H, D), dtype=torch.bfloat16, device=device), H * D, D
    else:
        n, h, d, ot, oh = _heads(out, "out", device)
        if (n, h, d) != (T, H, D):
            raise ValueError(f"out must be {(T, H, D)}, not {(n, h, d)}")
    lse = torch.empty((T, H), dtype=torch.float32, device=device) if return_lse else None
    _call(lib().pql_kv_attention, "kv_attention", device, KV_SCHEMES[cache.scheme], q.data_ptr(), qt, qh, T, H,
          *_cache_args(cache), cache.n_pages, cache.page_size, cache.n_kv_heads, D, starts.data_ptr(), lens.data_ptr(),
          pages.data_ptr(), B, width, ldp, causal, window, D ** -0.5 if scale is None else scale, out.data_ptr(), ot, oh,
          _ptr(lse), _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size())
    return (out, lse) if return_lse else out
