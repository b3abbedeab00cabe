"""PyTorch-facing helpers around the C ABI.

PyTorch provides device memory and streams; every step of the layer runs in
libcosmot's kernels.  These helpers only allocate outputs/workspace with torch
and translate tensors into the pointers and structs the C entry points take.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib as L

L.lib()  # the CUDA library must be present; no fallback


def ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def stream_handle(stream: Optional[torch.cuda.Stream] = None) -> int:
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libcosmot takes CUDA tensors only (no CPU fallback)")


WEIGHT_TENSORS = ("g1", "wqkv", "wo", "g2", "wg", "wu", "wd")


def weight_shapes(dims: L.Dims) -> dict:
    """Shape of every tensor of a layer's weight dict (row-major [out, in])."""
    d, f, hd = dims.d_model, dims.ffn, dims.head_dim
    per_set = {"g1": (d,), "wqkv": ((dims.n_heads + 2 * dims.n_kv_heads) * hd, d), "wo": (d, dims.n_heads * hd),
               "g2": (d,), "wg": (f, d), "wu": (f, d), "wd": (d, f)}
    shapes = {f"{s}.{t}": shp for s in ("R", "G") for t, shp in per_set.items()}
    shapes["gfin"] = (d,)
    shapes["wvel"] = (d, d)
    return shapes


def _check_bf16(t: torch.Tensor, name: str):
    if t.dtype != torch.bfloat16 or not t.is_contiguous():
        raise ValueError(f"{name}: libcosmot takes contiguous bf16 tensors (got {t.dtype}, "
                         f"{'contiguous' if t.is_contiguous() else 'strided'})")


def check_weights(dims: L.Dims, weights: dict):
    """The kernels read every weight through a bare pointer, so a tensor of the
    wrong shape, dtype or layout would be read out of bounds: refuse it here."""
    for name, shp in weight_shapes(dims).items():
        if name not in weights:
            raise ValueError(f"weight {name!r} missing")
        t = weights[name]
        if tuple(t.shape) != shp:
            raise ValueError(f"weight {name!r} has shape {tuple(t.shape)}, expected {shp}")
        _check_bf16(t, f"weight {name!r}")
    _need_cuda(*weights.values())


def _check_state(seq: L.SeqDesc, d: int, **ts):
    """h / h_out hold [batch][N][d] bf16 (N = n_ar + n_clean + n_noisy)."""
    rows = seq.batch * (seq.n_ar + seq.n_clean + seq.n_noisy)
    for name, t in ts.items():
        _check_bf16(t, name)
        if t.numel() < rows * d:
            raise ValueError(f"{name} holds {t.numel()} elements, fewer than batch x N x d = {rows * d}")
    _need_cuda(*ts.values())


def layout_spec(n_text: int, video=None, audio_clean=0, audio_noisy=0, audio_rate=25, action_clean=0,
                action_noisy=0, action_hz=15, proprio=0, tau_offset=0) -> L.LayoutSpec:
    """`video` = (views, grid_h, grid_w, fps, clean_steps, noisy_steps) or None."""
    v = video if video is not None else (0, 0, 0, 0, 0, 0)
    return L.LayoutSpec(n_text, *[int(x) for x in v], audio_clean, audio_noisy, audio_rate, action_clean,
                        action_noisy, action_hz, proprio, tau_offset)


@dataclass
class DeviceLayout:
    pos: torch.Tensor     # float32 [N, 3]
    chunk: torch.Tensor   # int32 [N]
    region: torch.Tensor  # int8 [N]
    n_ar: int
    n_clean: int
    n_noisy: int

    @property
    def n_tokens(self) -> int:
        return self.n_ar + self.n_clean + self.n_noisy


def build_layout(spec: L.LayoutSpec, device="cuda", stream=None) -> DeviceLayout:
    n, a, c, z = L.cosmot_layout_counts(spec)
    pos = torch.empty((n, 3), dtype=torch.float32, device=device)
    chunk = torch.empty((n,), dtype=torch.int32, device=device)
    region = torch.empty((n,), dtype=torch.int8, device=device)
    L.cosmot_build_layout(spec, ptr(pos), ptr(chunk), ptr(region), stream_handle(stream))
    return DeviceLayout(pos, chunk, region, a, c, z)


def mrope_table(pos: torch.Tensor, head_dim: int, sections, rope_base: float = 10000.0, stream=None) -> torch.Tensor:
    _need_cuda(pos)
    cs = torch.empty((pos.shape[0], head_dim // 2, 2), dtype=torch.float32, device=pos.device)
    L.cosmot_mrope_table(ptr(pos), pos.shape[0], head_dim, sections, rope_base, ptr(cs), stream_handle(stream))
    return cs


def make_dims(d_model, n_heads, n_kv_heads, head_dim, ffn, rope_sections, rope_base=10000.0, eps=1e-6) -> L.Dims:
    return L.Dims(d_model, n_heads, n_kv_heads, head_dim, ffn, (L.c_i32 * 3)(*rope_sections), rope_base, eps, 0)


class MoTLayer:
    """One MoT layer: both weight sets resident on the device.

    `weights` maps names to bf16 CUDA tensors: "R.*"/"G.*" for the Reasoner and
    Generator sets (g1, wqkv, wo, g2, wg, wu, wd), plus "gfin" and "wvel".
    """

    def __init__(self, dims: L.Dims, weights: dict):
        self.dims = dims
        self.weights = weights
        check_weights(dims, weights)
        sets = []
        for s in ("R", "G"):
            sets.append(L.SetWeights(*[ptr(weights[f"{s}.{t}"]) for t in ("g1", "wqkv", "wo", "g2", "wg", "wu", "wd")]))
        self.cw = L.LayerWeights((L.SetWeights * 2)(*sets), ptr(weights["gfin"]), ptr(weights["wvel"]))
        self._ws = None

    def seq_desc(self, n_ar, n_clean, n_noisy, batch, rope_cs, chunk=None, mask_mode=L.COSMOT_MASK_FULL,
                 n_cached=0) -> L.SeqDesc:
        """The descriptor holds raw pointers: rope_cs and chunk must stay alive while it is used."""
        return L.SeqDesc(n_ar, n_clean, n_noisy, batch, mask_mode, n_cached, ptr(rope_cs), ptr(chunk))

    def workspace_bytes(self, seq: L.SeqDesc) -> int:
        return L.cosmot_layer_workspace_size(self.dims, seq)

    def workspace(self, seq: L.SeqDesc, device="cuda") -> torch.Tensor:
        n = self.workspace_bytes(seq)
        if self._ws is None or self._ws.numel() < n:
            self._ws = torch.empty((n,), dtype=torch.uint8, device=device)
        return self._ws

    def commit_kv(self, h: torch.Tensor, seq: L.SeqDesc, dst_row: int, workspace: Optional[torch.Tensor] = None,
                  stream=None):
        """K/V of rows [seq.n_cached, N) of h into cache rows [dst_row, ...) of the workspace."""
        _check_state(seq, self.dims.d_model, h=h)
        ws = workspace if workspace is not None else self.workspace(seq, h.device)
        L.cosmot_layer_commit_kv(self.dims, self.cw, seq, ptr(h), dst_row, ptr(ws), ws.numel(), stream_handle(stream))

    def forward_cfg(self, h: torch.Tensor, h_out: torch.Tensor, sigma: float, sigma_next: float, guidance: float,
                    seq: L.SeqDesc, workspace: Optional[torch.Tensor] = None, stream=None):
        """Guided step: h [2P, N, d] holds (conditioned, baseline) pairs sharing their DM rows."""
        _check_state(seq, self.dims.d_model, h=h, h_out=h_out)
        ws = workspace if workspace is not None else self.workspace(seq, h.device)
        L.cosmot_layer_forward_cfg(self.dims, self.cw, seq, ptr(h), ptr(h_out), float(sigma), float(sigma_next),
                                   float(guidance), ptr(ws), ws.numel(), stream_handle(stream))

    def forward(self, h: torch.Tensor, h_out: torch.Tensor, sigma: float, sigma_next: float, seq: L.SeqDesc,
                workspace: Optional[torch.Tensor] = None, stream=None, x_state: Optional[torch.Tensor] = None,
                state_from_h: bool = False, vel: Optional[torch.Tensor] = None):
        """h [batch, N, d] bf16 (noisy DM rows updated in place to x'); h_out [batch, N, d] bf16.

        x_state: optional float32 [batch, n_noisy, d] sampler state of the noisy
        rows, read (unless state_from_h) and written in float32; h's noisy rows
        then receive its bf16 copy.  vel: optional bf16 [batch, n_noisy, d]
        receiving the velocity (see cosmot_layer_forward_io)."""
        _check_state(seq, self.dims.d_model, h=h, h_out=h_out)
        ws = workspace if workspace is not None else self.workspace(seq, h.device)
        io = self.step_io(seq, x_state, state_from_h, vel)
        if io is None:
            L.cosmot_layer_forward(self.dims, self.cw, seq, ptr(h), ptr(h_out), float(sigma), float(sigma_next),
                                   ptr(ws), ws.numel(), stream_handle(stream))
        else:
            L.cosmot_layer_forward_io(self.dims, self.cw, seq, ptr(h), ptr(h_out), float(sigma), float(sigma_next),
                                      io, ptr(ws), ws.numel(), stream_handle(stream))

    def step_io(self, seq: L.SeqDesc, x_state: Optional[torch.Tensor] = None, state_from_h: bool = False,
                vel: Optional[torch.Tensor] = None) -> Optional[L.StepIO]:
        """The StepIO struct for an optional float32 state and velocity output,
        both [batch, n_noisy, d] contiguous (checked here: the kernels read and
        write them through bare pointers)."""
        if x_state is None and vel is None:
            return None
        d, rows = self.dims.d_model, seq.batch * seq.n_noisy
        for name, t, dt in (("x_state", x_state, torch.float32), ("vel", vel, torch.bfloat16)):
            if t is None:
                continue
            _need_cuda(t)
            if t.dtype != dt or not t.is_contiguous() or t.numel() < rows * d:
                raise ValueError(f"{name}: expected a contiguous {dt} tensor of batch x n_noisy x d = {rows * d} "
                                 f"elements (got {t.dtype}, {t.numel()})")
        return L.step_io(ptr(x_state), d, ptr(vel), d, state_from_h)


class MoTStack:
    """A stack of MoT layers with one velocity head (that of the last layer).

    `layers` is a list of weight dicts as MoTLayer takes (bf16 CUDA tensors);
    the same dict may appear more than once.
    """

    def __init__(self, dims: L.Dims, layers: list):
        self.dims = dims
        self.layers = [MoTLayer(dims, w) for w in layers]
        self.cw = (L.LayerWeights * len(self.layers))(*[m.cw for m in self.layers])
        self._ws = None

    def seq_desc(self, *args, **kw) -> L.SeqDesc:
        return self.layers[0].seq_desc(*args, **kw)

    def workspace_bytes(self, seq: L.SeqDesc) -> int:
        return L.cosmot_stack_workspace_size(self.dims, len(self.layers), seq)

    def workspace(self, seq: L.SeqDesc, device="cuda") -> torch.Tensor:
        n = self.workspace_bytes(seq)
        if self._ws is None or self._ws.numel() < n:
            self._ws = torch.empty((n,), dtype=torch.uint8, device=device)
        return self._ws

    def forward(self, h: torch.Tensor, h_out: torch.Tensor, sigma: float, sigma_next: float, seq: L.SeqDesc,
                workspace: Optional[torch.Tensor] = None, stream=None, x_state: Optional[torch.Tensor] = None,
                state_from_h: bool = False, vel: Optional[torch.Tensor] = None):
        """h^L into h_out; x' into the noisy rows of h (see cosmot_stack_forward);
        x_state / vel as for MoTLayer.forward."""
        _check_state(seq, self.dims.d_model, h=h, h_out=h_out)
        ws = workspace if workspace is not None else self.workspace(seq, h.device)
        io = self.layers[0].step_io(seq, x_state, state_from_h, vel)
        if io is None:
            L.cosmot_stack_forward(self.dims, self.cw, seq, ptr(h), ptr(h_out), sigma, sigma_next, ptr(ws),
                                   ws.numel(), stream_handle(stream))
        else:
            L.cosmot_stack_forward_io(self.dims, self.cw, seq, ptr(h), ptr(h_out), sigma, sigma_next, io, ptr(ws),
                                      ws.numel(), stream_handle(stream))


def _rows_layout(t: torch.Tensor, name: str, batch: int, heads: Optional[int], head_dim: int, dtype, n: Optional[int] = None):
    """(ld, rows between sequences) of a [batch, n, heads, head_dim] tensor whose
    rows hold their heads side by side; a view of a wider row (the columns of a
    QKV projection) fits."""
    if t.dtype is dtype and t.dim() == 4:  # the usual tensor, without the detours below
        b, rows, h, hd = t.shape
        s0, s1, s2, s3 = t.stride()
        if b == batch and hd == head_dim and (h == heads or heads is None) and (rows == n or n is None) and s3 == 1 and \
                h > 0 and (s2 == hd or h == 1):
            if rows == 1 and (s0 >= h * hd or batch == 1):
                return (s0, 1) if batch > 1 else (h * hd, 1)
            if rows > 1 and s1 >= h * hd:
                if batch == 1:
                    return s1, rows
                if s0 % s1 == 0 and s0 >= rows * s1:
                    return s1, s0 // s1
    if t.dim() != 4 or t.shape[0] != batch or t.shape[3] != head_dim or (heads is not None and t.shape[2] != heads) or \
            (n is not None and t.shape[1] != n):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [{batch}, {'n' if n is None else n}, "
                         f"{'heads' if heads is None else heads}, {head_dim}]")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    h, rows = t.shape[2], t.shape[1]
    s0, s1, s2, s3 = t.stride()
    width = h * head_dim
    if t.numel() == 0:
        return width, rows
    if s3 != 1 or (h > 1 and s2 != head_dim):
        raise ValueError(f"{name}: a row's heads must lie side by side (strides {t.stride()})")
    if rows == 1:  # the stride of a dimension of one says nothing
        ld, between = (s0, 1) if batch > 1 else (width, 1)
    else:
        ld, between = s1, rows
        if batch > 1:
            if ld <= 0 or s0 % ld:
                raise ValueError(f"{name}: the batch stride must be a whole number of rows (strides {t.stride()})")
            between = s0 // ld
    if ld < width or between < rows:
        raise ValueError(f"{name}: rows overlap (strides {t.stride()})")
    return ld, between


class KVCache8:
    """A key/value cache in 8 bits: e4m3 rows with one float32 scale for each
    block of rows and key head (see cosmot_kv8_cache).

    Wraps the caller's tensors: k, v float8_e4m3fn [batch, capacity, n_kv_heads,
    head_dim]; k_scale, v_scale float32 [batch, n_kv_heads, blocks], blocks =
    ceil(capacity / block); lens int32 [batch], the rows each sequence holds.
    `KVCache8.empty` makes them.  A streaming step:

        cache.store(k, v)                              # behind the rows held
        o, lse = cache.attend(q, n_new=n)              # over them and the new ones
        cache.weigh(q, lse, weight, n_new=n)           # optional: what got attention
        cache.advance(n)                               # after the last denoising step
        cache.evict(weight, keep_blocks, first_rows=n_ar, last_rows=n)

    Every call, advance too, runs on `stream` (default: the current one of the
    cache's device) and follows `lens` on the device, so it may be captured into a
    CUDA graph.  On another stream a call first waits for what the current one has
    been given so far.  Outputs and workspaces that a call makes are its own.  A
    workspace given by the caller serves one call at a time.
    The library reports lengths outside the cache through the device status.
    The tensors stay the ones that the cache was made with (its kernels and captured
    graphs go by their addresses): write into them, `lens.copy_(...)`.
    """

    _FIXED = frozenset(("k", "v", "k_scale", "v_scale", "lens", "block", "batch", "capacity", "n_kv_heads", "head_dim", "n_blocks",
                        "device"))

    def __setattr__(self, name, value):
        if name in self._FIXED and hasattr(self, "desc") and value is not getattr(self, name):  # (lens += n is in place)
            raise AttributeError(f"KVCache8.{name} is what the cache was made with; write into its tensors instead of replacing them")
        super().__setattr__(name, value)

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                 lens: torch.Tensor, block: int):
        _need_cuda(k, v, k_scale, v_scale, lens)
        if k.dim() != 4:
            raise ValueError(f"k has shape {tuple(k.shape)}, expected [batch, capacity, n_kv_heads, head_dim]")
        batch, capacity, n_kv, hd = k.shape
        if block not in (16, 32, 64, 128):
            raise ValueError(f"block {block}: 16, 32, 64 or 128")
        layout = _rows_layout(k, "k", batch, n_kv, hd, torch.float8_e4m3fn)
        if _rows_layout(v, "v", batch, n_kv, hd, torch.float8_e4m3fn, capacity) != layout:
            raise ValueError("k and v must have the same strides")
        self.n_blocks = -(-capacity // block)
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            self._check(name, t, torch.float32, (batch, n_kv, self.n_blocks))
        self._check("lens", lens, torch.int32, (batch,))
        if len({t.device for t in (k, v, k_scale, v_scale, lens)}) != 1:
            raise ValueError("the cache's tensors must be on one device")
        self.k, self.v, self.k_scale, self.v_scale, self.lens, self.block = k, v, k_scale, v_scale, lens, block
        self.batch, self.capacity, self.n_kv_heads, self.head_dim = batch, capacity, n_kv, hd
        self.device = k.device
        self.desc = L.Kv8Cache(ptr(k), ptr(v), ptr(k_scale), ptr(v_scale), ptr(lens), layout[0], layout[1], batch,
                               capacity, n_kv, hd, block, 0)
        self._ref = ctypes.byref(self.desc)
        self._plans = {}
        self._one = {t: torch.empty((1,), dtype=t, device=self.device) for t in (torch.bfloat16, torch.float32, torch.uint8)}
        self._evict_like = None

    @classmethod
    def empty(cls, batch: int, capacity: int, n_kv_heads: int, head_dim: int, block: int = 64, device="cuda"):
        rows = lambda: torch.zeros((batch, capacity, n_kv_heads, head_dim), dtype=torch.uint8,  # noqa: E731
                                   device=device).view(torch.float8_e4m3fn)
        scales = lambda: torch.ones((batch, n_kv_heads, -(-capacity // block)), device=device)  # noqa: E731
        return cls(rows(), rows(), scales(), scales(), torch.zeros((batch,), dtype=torch.int32, device=device), block)

    def empty_weight(self) -> torch.Tensor:
        """Accumulated weights for weigh / evict, all zero."""
        return torch.zeros((self.batch, self.n_kv_heads, self.n_blocks), device=self.device)

    @staticmethod
    def _check(name, t, dtype, shape):
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} (got {t.dtype}, "
                             f"{tuple(t.shape)}, {'contiguous' if t.is_contiguous() else 'strided'})")

    def _here(self, name: str, t: torch.Tensor):
        if t.get_device() != self.device.index:
            raise ValueError(f"{name} is on {t.device}, the cache on {self.device}")

    def _stream(self, stream, *made) -> int:
        """The stream's handle.  Another stream than the current one first waits for that one, which
        may still write the inputs and owns the memory of tensors made here; they are kept until the
        other is done."""
        if stream is None:  # torch.cuda.current_stream(device).cuda_stream, without the object
            return torch._C._cuda_getCurrentRawStream(self.device.index)
        if stream.device != self.device:
            raise ValueError(f"the stream is on {stream.device}, the cache on {self.device}")
        current = torch.cuda.current_stream(self.device)
        if current != stream:
            stream.wait_stream(current)
            for t in made:
                if t is not None:
                    t.record_stream(stream)
        return stream.cuda_stream

    def _call(self, name: str, *args):
        """One of the library's entries, on the cache's device."""
        fn = getattr(L.lib(), name)
        if torch.cuda.current_device() == self.device.index:
            code = fn(self._ref, *args)
        else:
            with torch.cuda.device(self.device):
                code = fn(self._ref, *args)
        if code != L.COSMOT_OK:
            raise L.CosmotError(name, code)

    def _shape(self, shape, dtype):
        """One element seen as a tensor of `shape`: torch.empty_like gives a new contiguous one."""
        return self._one[dtype].expand(shape)

    def _workspace(self, need: int, like: Optional[torch.Tensor], workspace: Optional[torch.Tensor]):
        """(tensor, made here): the caller's workspace, or one for this call."""
        if workspace is not None:
            self._here("workspace", workspace)
            if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.numel() < need:
                raise ValueError(f"workspace: expected at least {need} contiguous uint8 elements")
            return workspace, None
        made = torch.empty_like(like, memory_format=torch.contiguous_format) if need else None
        return made, made

    def _query(self, q: torch.Tensor, n_new: int, causal: bool, max_len: int, softmax_scale: float, o_between: int = 0):
        """(descriptor, elements between q's rows, attention's workspace bytes, and the
        shapes of o, lse and the workspace).  They depend on sizes and strides alone and
        are kept for calls of the same ones."""
        key = (q.shape, q.stride(), q.dtype, o_between, n_new, causal, max_len, softmax_scale)
        plan = self._plans.get(key)
        if plan is None:
            ld, between = _rows_layout(q, "q", self.batch, None, self.head_dim, torch.bfloat16)
            self._here("q", q)
            _, n, heads, hd = q.shape
            desc = L.Kv8Query(n, between, o_between or n, heads, n_new, L.COSMOT_KV8_CAUSAL if causal else L.COSMOT_KV8_FULL,
                              max_len, softmax_scale, 0)
            need = ctypes.c_size_t(0)
            self._call("cosmot_kv8_attention_workspace", ctypes.byref(desc), ctypes.byref(need))
            if len(self._plans) >= 64:
                self._plans = {}
            plan = self._plans[key] = (ctypes.byref(desc), ld, need.value, self._shape(q.shape, torch.bfloat16),
                                       self._shape((self.batch, heads, n), torch.float32),
                                       self._shape((need.value,), torch.uint8))
        self._here("q", q)
        return plan

    def advance(self, n: int, stream=None):
        """The last n stored rows become rows held."""
        if stream is None:
            self.lens.add_(n)
            return
        self._stream(stream)
        with torch.cuda.stream(stream):
            self.lens.add_(n)

    def store(self, k: torch.Tensor, v: torch.Tensor, stream=None):
        """Rows [batch, n, n_kv_heads, head_dim] (bf16, views of a QKV projection
        fit) behind the ones held; `advance` makes them held."""
        n = k.shape[1] if k.dim() == 4 else None
        ld, between = _rows_layout(k, "k", self.batch, self.n_kv_heads, self.head_dim, torch.bfloat16)
        if _rows_layout(v, "v", self.batch, self.n_kv_heads, self.head_dim, torch.bfloat16, n) != (ld, between):
            raise ValueError("k and v must have the same strides")
        self._here("k", k)
        self._here("v", v)
        if n:
            self._call("cosmot_kv8_store", k.data_ptr(), v.data_ptr(), ld, between, n, self._stream(stream))

    def attend(self, q: torch.Tensor, n_new: int = 0, causal: bool = False, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, max_len: int = 0, softmax_scale: float = 0.0,
               workspace: Optional[torch.Tensor] = None, stream=None):
        """(o, lse) of q [batch, n, n_heads, head_dim] bf16 over the rows held and
        n_new more: o as q, lse float32 [batch, n_heads, n] (natural log).  causal:
        query i is row len - n + i and sees the rows up to itself; otherwise every
        row.  max_len: the most rows any sequence shows, if known (it sizes the
        split of the work only)."""
        if q.dim() != 4:
            raise ValueError(f"q has shape {tuple(q.shape)}, expected [batch, n, heads, head_dim]")
        batch, n, heads, hd = q.shape
        o_between = 0
        if out is not None:
            ld_o, o_between = _rows_layout(out, "out", self.batch, heads, self.head_dim, torch.bfloat16, n)
            self._here("out", out)
        if lse is not None:
            self._check("lse", lse, torch.float32, (batch, heads, n))
            self._here("lse", lse)
        desc, ld, need, like_o, like_lse, like_ws = self._query(q, n_new, causal, max_len, softmax_scale, o_between)
        made = []
        if out is None:
            out, ld_o = torch.empty_like(like_o, memory_format=torch.contiguous_format), heads * hd
            made.append(out)
        if lse is None:
            lse = torch.empty_like(like_lse, memory_format=torch.contiguous_format)
            made.append(lse)
        if n == 0:
            return out, lse
        ws, fresh = self._workspace(need, like_ws, workspace)
        self._call("cosmot_kv8_attention", desc, q.data_ptr(), ld, out.data_ptr(), ld_o, lse.data_ptr(), ptr(ws),
                   0 if ws is None else ws.numel(), self._stream(stream, *made, fresh))
        return out, lse

    def weigh(self, q: torch.Tensor, lse: torch.Tensor, weight: torch.Tensor, decay: float = 1.0, n_new: int = 0,
              causal: bool = False, max_len: int = 0, softmax_scale: float = 0.0, stream=None) -> torch.Tensor:
        """weight [batch, n_kv_heads, blocks] = decay * weight + the attention
        weight of q's rows for each block; lse as `attend` gave it for the same
        query.  Returns weight."""
        desc, ld, *_ = self._query(q, n_new, causal, max_len, softmax_scale)
        self._check("lse", lse, torch.float32, (self.batch, q.shape[2], q.shape[1]))
        self._check("weight", weight, torch.float32, (self.batch, self.n_kv_heads, self.n_blocks))
        self._here("lse", lse)
        self._here("weight", weight)
        if q.shape[1] == 0:
            raise ValueError("weigh needs at least one query")
        self._call("cosmot_kv8_weigh", desc, q.data_ptr(), ld, lse.data_ptr(), decay, weight.data_ptr(), self._stream(stream))
        return weight

    def evict(self, weight: torch.Tensor, keep_blocks: int, first_rows: int = 0, last_rows: int = 0,
              in_place: bool = True, workspace: Optional[torch.Tensor] = None, stream=None):
        """Brings every sequence and key head down to keep_blocks blocks of rows:
        the ones that hold the first first_rows or the last last_rows rows, or a
        part of a block, then those of the most weight.  The cache's rows and
        scales move up in place; (weight, lens) follow in place too, or, with
        in_place=False, are returned as new tensors: the cache then still goes by
        the old lengths, and is not to be used before the new ones are copied into
        `lens`."""
        self._check("weight", weight, torch.float32, (self.batch, self.n_kv_heads, self.n_blocks))
        self._here("weight", weight)
        w_out, lens = (weight, self.lens) if in_place else (torch.empty_like(weight), torch.empty_like(self.lens))
        if self._evict_like is None:
            self._evict_like = self._shape((L.cosmot_kv8_evict_workspace(self.desc),), torch.uint8)
        ws, fresh = self._workspace(self._evict_like.numel(), self._evict_like, workspace)
        made = (fresh,) if in_place else (fresh, w_out, lens)
        self._call("cosmot_kv8_evict", weight.data_ptr(), keep_blocks, first_rows, last_rows, w_out.data_ptr(),
                   lens.data_ptr(), ws.data_ptr(), ws.numel(), self._stream(stream, *made))
        return w_out, lens
