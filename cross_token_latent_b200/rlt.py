"""Python binding of librlt.so (the C ABI in include/rlt.h).

Argument marshalling only: PyTorch provides device memory and the current CUDA
stream; every step of the encoder, the decoder transition and the replay runs in
the library's kernels.  There is no CPU or PyTorch fallback: if the library is
missing or no CUDA device is present, the calls raise.
"""
from __future__ import annotations

import ctypes
from pathlib import Path

import numpy as np
import torch

LIB_PATH = Path(__file__).resolve().parent / "librlt.so"

RLT_F32, RLT_BF16 = 0, 1
STATUS = {0: "RLT_OK", 1: "RLT_EINVAL", 2: "RLT_ECUDA", 3: "RLT_ESTALE", 4: "RLT_ETIMEOUT",
          5: "RLT_EUNSUPPORTED", 6: "RLT_EDEVICE", 7: "RLT_ESTATE"}


class RLTError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        self.status = STATUS.get(code, str(code))
        super().__init__(f"{what}: {self.status}")


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("V", "d", "n_heads", "head_dim", "L_E", "L_D", "F", "W", "G",
                                                "dtype")] + \
               [("rms_eps", ctypes.c_float), ("rope_base", ctypes.c_float), ("max_pos", ctypes.c_int32)]


class PagedBatchArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "N", "max_q", "max_kv")] + \
               [(n, ctypes.c_void_p) for n in ("q_start", "kv_len", "table")] + \
               [(n, ctypes.c_int32) for n in ("table_stride", "page_size", "n_pages", "n_kv_heads")]


class LogitsArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("out_stride", ctypes.c_int64), ("lse", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("bias_stride", ctypes.c_int64), ("mask", ctypes.c_void_p), ("mask_stride", ctypes.c_int64),
                ("tokens", ctypes.c_void_p), ("seq_stride", ctypes.c_int64), ("tok_stride", ctypes.c_int64),
                ("n_tokens", ctypes.c_int32), ("tok_len", ctypes.c_void_p), ("gen_start", ctypes.c_void_p),
                ("repetition", ctypes.c_void_p), ("presence", ctypes.c_void_p), ("frequency", ctypes.c_void_p),
                ("tau", ctypes.c_void_p), ("out_lse", ctypes.c_void_p)]


_lib = None
_EXPORTS = {
    "rlt_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "rlt_weights_bytes": (ctypes.c_size_t, [ctypes.POINTER(Config)]),
    "rlt_model_create": (ctypes.c_int, [ctypes.POINTER(Config), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                        ctypes.POINTER(ctypes.c_void_p)]),
    "rlt_model_destroy": (None, [ctypes.c_void_p]),
    "rlt_model_set_weight": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_char_p, ctypes.c_void_p, ctypes.c_size_t,
                                            ctypes.c_void_p]),
    "rlt_model_commit": (ctypes.c_int, [ctypes.c_void_p]),
    "rlt_model_version": (ctypes.c_uint64, [ctypes.c_void_p]),
    "rlt_encode_workspace_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int]),
    "rlt_encode": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                  ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                  ctypes.c_void_p]),
    "rlt_encoder_cache_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int]),
    "rlt_encode_prefill": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                          ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "rlt_encode_append_workspace_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int]),
    "rlt_encode_append": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t,
                                         ctypes.c_void_p]),
    "rlt_sample": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int,
                                  ctypes.c_float, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "rlt_page_pool_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "rlt_paged_append": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                        ctypes.c_void_p]),
    "rlt_paged_attention_workspace_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int]),
    "rlt_paged_attention": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_int64,
                                           ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "rlt_encode_chunk_workspace_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_void_p]),
    "rlt_encode_chunk": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                        ctypes.c_size_t, ctypes.c_void_p]),
    "rlt_process_logits": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]),
    "rlt_state_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int]),
    "rlt_state_positions_offset": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int]),
    "rlt_state_positions": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(ctypes.c_int64)]),
    "rlt_state_reset_row": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]),
    "rlt_snapshot_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int]),
    "rlt_snapshot_save": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int,
                                         ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t,
                                         ctypes.c_void_p]),
    "rlt_snapshot_load": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                         ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int,
                                         ctypes.c_void_p]),
    "rlt_state_init": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]),
    "rlt_state_copy": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "rlt_state_position": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(ctypes.c_int64)]),
    "rlt_state_release": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "rlt_decode_workspace_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int]),
    "rlt_decode_step": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_float,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_size_t, ctypes.c_void_p]),
    "rlt_decode_step_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                               ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_float,
                                               ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                               ctypes.c_void_p]),
    "rlt_replay_workspace_bytes": (ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int]),
    "rlt_replay": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                  ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                  ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "rlt_last_error": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "rlt_launch_count": (ctypes.c_uint64, [ctypes.c_void_p]),
    "rlt_gemm_bf16": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "rlt_gemm_plan": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "rlt_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                                 ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                 ctypes.c_uint64, ctypes.c_void_p]),
    "rlt_set_option": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_char_p, ctypes.c_int64]),
    "rlt_profile_start": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_uint32]),
    "rlt_profile_stop": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_double),
                                        ctypes.POINTER(ctypes.c_uint64)]),
}

KERNEL_KINDS = ["norm", "merge", "qkv", "swa", "o_proj", "qc_proj", "xattn", "oc_proj", "ffn_up", "ffn_down",
                "final_norm", "head", "lse", "encoder", "small_step", "enc_gemm", "enc_attn", "enc_other"]


def lib() -> ctypes.CDLL:
    """Load librlt.so (raises if it was never built)."""
    global _lib
    if _lib is None:
        if not LIB_PATH.exists():
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m cross_token_latent_b200.build`")
        h = ctypes.CDLL(str(LIB_PATH))
        for name, (res, args) in _EXPORTS.items():
            f = getattr(h, name)
            f.restype = res
            f.argtypes = args
        _lib = h
    return _lib


def exported_names() -> list[str]:
    return list(_EXPORTS)


def gemm_plan(M: int, N: int, K: int) -> int:
    """Kernel id (as rlt_gemm_bf16 numbers them) the library picks for an M x N x K bf16 product."""
    return lib().rlt_gemm_plan(M, N, K)


def _check(code: int, what: str) -> None:
    if code != 0:
        raise RLTError(code, what)


def _ptr(t) -> ctypes.c_void_p | None:
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream() -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def make_config(cfg, max_pos: int) -> Config:
    """cfg: any object with the ModelConfig fields (V, d, n_heads, ..., dtype 'f32'|'bf16')."""
    return Config(cfg.V, cfg.d, cfg.n_heads, cfg.head_dim, cfg.L_E, cfg.L_D, cfg.F, cfg.W, cfg.G,
                  RLT_BF16 if cfg.dtype == "bf16" else RLT_F32, float(cfg.rms_eps), float(cfg.rope_base),
                  int(max_pos))


class RLTState:
    """A caller-owned decoder state buffer H (registered with its model)."""

    def __init__(self, model: "RLTModel", B: int, buf: torch.Tensor):
        self.model, self.B, self.buf = model, B, buf

    @property
    def position(self) -> int:
        t = ctypes.c_int64()
        _check(lib().rlt_state_position(self.model.handle, _ptr(self.buf), ctypes.byref(t)), "rlt_state_position")
        return t.value

    def s(self) -> torch.Tensor:
        """View of s_t [B, d] float32 inside the state buffer."""
        d = self.model.cfg.d
        return self.buf[256:256 + self.B * d * 4].view(torch.float32).view(self.B, d)

    def positions(self) -> list[int]:
        """Tokens consumed by every sequence (host registry)."""
        out = (ctypes.c_int64 * self.B)()
        _check(lib().rlt_state_positions(self.model.handle, _ptr(self.buf), out), "rlt_state_positions")
        return list(out)

    def positions_device(self) -> torch.Tensor:
        """View of the state's int32 [B] device positions (what rlt_encode_append takes)."""
        off = lib().rlt_state_positions_offset(self.model.handle, self.B)
        return self.buf[off:off + 4 * self.B].view(torch.int32)

    def reset_row(self, row: int) -> None:
        _check(lib().rlt_state_reset_row(self.model.handle, _ptr(self.buf), int(row), _stream()), "rlt_state_reset_row")

    def copy(self) -> "RLTState":
        other = torch.empty_like(self.buf)
        _check(lib().rlt_state_copy(self.model.handle, _ptr(other), _ptr(self.buf), _stream()), "rlt_state_copy")
        return RLTState(self.model, self.B, other)

    def __del__(self):
        try:
            if self.model.handle:
                lib().rlt_state_release(self.model.handle, _ptr(self.buf))
        except Exception:
            pass


def _need(t: torch.Tensor, what: str, dtype, device: int, shape: tuple) -> None:
    """ValueError unless t is a tensor of this type and shape on CUDA device number `device`."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape:
        raise ValueError(f"{what}: need {dtype} {list(shape)} on cuda:{device}, got {t.dtype} {list(t.shape)} on {t.device}")


def _rows(t: torch.Tensor, what: str, dtype, device: int, shape: tuple) -> tuple[int, int]:
    """(address, elements between rows) of a tensor of this type and shape [N, heads, head_dim], whose
    rows are contiguous."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape:
        _need(t, what, dtype, device, shape)
    s0, s1, s2 = t.stride()
    n, h, d = shape
    if s2 != 1 or (s1 != d and h > 1):
        raise ValueError(f"{what}: the heads of a row must be contiguous")
    return t.data_ptr(), s0 if n > 1 else h * d


class PagedBatch:
    """The new tokens of a ragged batch over a paged key/value cache (rlt_paged_batch in
    include/rlt.h): its device arrays and the bounds the host knows.  Made once and used for every
    layer; what the device arrays hold may change between calls."""

    def __init__(self, model: "RLTModel", table: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor, N: int,
                 max_q: int, max_kv: int, page_size: int, n_kv_heads: int):
        B = kv_len.shape[0]
        _need(table, "table", torch.int32, model._dev, (B, table.shape[-1]))
        _need(q_start, "q_start", torch.int32, model._dev, (B + 1,))
        _need(kv_len, "kv_len", torch.int32, model._dev, (B,))
        if not (q_start.is_contiguous() and kv_len.is_contiguous()) or table.stride(1) != 1 or \
                table.stride(0) < table.shape[1]:
            raise ValueError("q_start, kv_len and the rows of the page table must be contiguous")
        cols = table.shape[1]
        if not (1 <= max_q <= N and max_q <= max_kv <= min(model.max_pos, cols * page_size)):
            raise ValueError(f"need 1 <= max_q <= N and max_q <= max_kv <= min(max_pos, {cols} pages): "
                             f"got N {N}, max_q {max_q}, max_kv {max_kv}")
        self.model, self.B, self.N = model, B, int(N)
        self.page_size, self.n_kv_heads = int(page_size), int(n_kv_heads)
        self.table, self.q_start, self.kv_len = table, q_start, kv_len
        self.c = PagedBatchArgs(B, int(N), int(max_q), int(max_kv), q_start.data_ptr(), kv_len.data_ptr(),
                                table.data_ptr(), table.stride(0) if B > 1 else cols, int(page_size), 0,
                                int(n_kv_heads))
        self.ref = ctypes.byref(self.c)
        self._page = (2, self.n_kv_heads, self.page_size, model.cfg.head_dim)
        self._ws: dict = {}                        # workspace bytes by (n_pages, n_heads)

    def args(self, pool: torch.Tensor):
        """The C structure for calls on this pool [n_pages, 2, n_kv_heads, page_size, head_dim]."""
        n = pool.shape[0]
        _need(pool, "pool", self.model.sdtype, self.model._dev, (n, *self._page))
        if not pool.is_contiguous():
            raise ValueError("pool: must be contiguous")
        self.c.n_pages = n
        return self.ref

    def attention_workspace_bytes(self, n_heads: int) -> int:
        key = (self.c.n_pages, n_heads)
        nb = self._ws.get(key)
        if nb is None:
            nb = self._ws[key] = lib().rlt_paged_attention_workspace_bytes(self.model.handle, self.ref, n_heads)
        return nb


class RLTModel:
    """One model on one CUDA device: weight arena, encoder, decoder step and replay."""

    def __init__(self, cfg, max_pos: int, device: str | torch.device = "cuda"):
        if not torch.cuda.is_available():
            raise RuntimeError("RLTModel needs a CUDA device")
        self.cfg = cfg
        self.device = torch.device(device)
        if self.device.index is None:
            self.device = torch.device(self.device.type, torch.cuda.current_device())
        self._dev = self.device.index
        self.max_pos = int(max_pos)
        self.sdtype = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
        self._c = make_config(cfg, max_pos)
        nbytes = lib().rlt_weights_bytes(ctypes.byref(self._c))
        if nbytes == 0:
            raise RLTError(1, "rlt_weights_bytes (config rejected)")
        self.arena = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        h = ctypes.c_void_p()
        _check(lib().rlt_model_create(ctypes.byref(self._c), _ptr(self.arena), nbytes, _stream(), ctypes.byref(h)),
               "rlt_model_create")
        self.handle = h
        self._ws: dict = {}
        self._destroy = lib().rlt_model_destroy    # held so that teardown at exit still reaches it

    def __del__(self):
        h = getattr(self, "handle", None)
        destroy = getattr(self, "_destroy", None)
        if h and destroy is not None:
            destroy(h)
            self.handle = None

    # ---------------------------------------------------------------- weights
    def set_weight(self, name: str, value) -> None:
        t = torch.as_tensor(np.ascontiguousarray(value, dtype=np.float32) if isinstance(value, np.ndarray) else value)
        t = t.to(device=self.device, dtype=torch.float32).contiguous()
        _check(lib().rlt_model_set_weight(self.handle, name.encode(), _ptr(t), t.numel(), _stream()),
               f"rlt_model_set_weight({name})")
        self._keep = t     # the copy is stream-ordered; keep the source alive until the next call

    def load_weights(self, weights: dict) -> None:
        for name, value in weights.items():
            self.set_weight(name, value)
        _check(lib().rlt_model_commit(self.handle), "rlt_model_commit")
        torch.cuda.current_stream().synchronize()
        self._keep = None

    def set_option(self, name: str, value: int) -> None:
        """Scheduling option of the handle (rlt_set_option): "row_groups", "group_attn_ctas_per_sm",
        "group_pdl"."""
        _check(lib().rlt_set_option(self.handle, name.encode(), int(value)), f"rlt_set_option({name})")

    @property
    def version(self) -> int:
        return lib().rlt_model_version(self.handle)

    @property
    def launch_count(self) -> int:
        return lib().rlt_launch_count(self.handle)

    def _raw_stream(self) -> int:
        """The current stream of the model's device, as the C ABI takes it."""
        return torch._C._cuda_getCurrentRawStream(self._dev)

    def _workspace(self, key, nbytes: int) -> torch.Tensor:
        buf = self._ws.get(key)
        if buf is None or buf.numel() < nbytes:
            buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
            self._ws[key] = buf
        return buf

    def release_workspaces(self) -> None:
        self._ws.clear()

    # ---------------------------------------------------------------- encoder
    def alloc_encoder_outputs(self, B: int, T_alloc: int):
        c = self.cfg
        e = torch.empty((B, T_alloc, c.d), dtype=self.sdtype, device=self.device)
        M = torch.empty((c.G, 2, B, c.n_heads, T_alloc, c.head_dim), dtype=self.sdtype, device=self.device)
        return e, M

    def encode(self, tokens: torch.Tensor, T_alloc: int | None = None, out=None):
        """tokens int32 [B, T] on the device -> (e [B, T_alloc, d], M [G, 2, B, H, T_alloc, hd])."""
        tokens = tokens.to(device=self.device, dtype=torch.int32).contiguous()
        B, T = tokens.shape
        T_alloc = T if T_alloc is None else T_alloc
        e, M = out if out is not None else self.alloc_encoder_outputs(B, T_alloc)
        nb = lib().rlt_encode_workspace_bytes(self.handle, B, T)
        ws = self._workspace(("enc", B, T), nb)
        _check(lib().rlt_encode(self.handle, _ptr(tokens), B, T, T_alloc, _ptr(e), _ptr(M), _ptr(ws), ws.numel(),
                                _stream()), "rlt_encode")
        return e, M

    # ---------------------------------------------------------------- incremental encoder
    def alloc_encoder_cache(self, B: int, T_max: int) -> torch.Tensor:
        return torch.empty(lib().rlt_encoder_cache_bytes(self.handle, B, T_max), dtype=torch.uint8,
                           device=self.device)

    def encode_prefill(self, tokens: torch.Tensor, T_alloc: int, T_max: int | None = None, out=None, cache=None):
        """rlt_encode_prefill: (e, M, encoder cache) of the first T tokens, capacities T_alloc / T_max."""
        tokens = tokens.to(device=self.device, dtype=torch.int32).contiguous()
        B, T = tokens.shape
        T_max = T_alloc if T_max is None else T_max
        e, M = out if out is not None else self.alloc_encoder_outputs(B, T_alloc)
        cache = self.alloc_encoder_cache(B, T_max) if cache is None else cache
        nb = lib().rlt_encode_workspace_bytes(self.handle, B, T)
        ws = self._workspace(("enc", B, T), nb)
        _check(lib().rlt_encode_prefill(self.handle, _ptr(tokens), B, T, T_alloc, _ptr(e), _ptr(M), _ptr(cache), T_max,
                                        _ptr(ws), ws.numel(), _stream()), "rlt_encode_prefill")
        return e, M, cache

    def encode_append(self, tokens: torch.Tensor, pos: int, cache: torch.Tensor, T_max: int, e: torch.Tensor,
                      M: torch.Tensor, positions: torch.Tensor | None = None) -> None:
        """rlt_encode_append: tokens is an int32 device vector [B] or a column view of a [B, T]
        matrix (its stride is passed through); the token at position pos is encoded, or with
        `positions` (int32 device [B], e.g. RLTState.positions_device()) sequence b's token at
        positions[b] <= pos."""
        B = tokens.shape[0]
        stride = tokens.stride(0)
        nb = lib().rlt_encode_append_workspace_bytes(self.handle, B)
        ws = self._workspace(("app", B), nb)
        _check(lib().rlt_encode_append(self.handle, _ptr(tokens), stride, B, int(pos), _ptr(positions), _ptr(cache),
                                       int(T_max), _ptr(e), _ptr(M), e.shape[1], _ptr(ws), ws.numel(), _stream()),
               "rlt_encode_append")

    # ---------------------------------------------------------------- sequence snapshots
    def snapshot_save(self, state: "RLTState", row: int, M: torch.Tensor, cache: torch.Tensor | None = None,
                      T_max: int = 0) -> torch.Tensor:
        """rlt_snapshot_save of sequence `row` into a new device buffer."""
        t = state.positions()[row]
        buf = torch.empty(lib().rlt_snapshot_bytes(self.handle, t), dtype=torch.uint8, device=self.device)
        _check(lib().rlt_snapshot_save(self.handle, _ptr(state.buf), int(row), _ptr(cache), int(T_max), _ptr(M),
                                       M.shape[4], _ptr(buf), buf.numel(), _stream()), "rlt_snapshot_save")
        return buf

    def snapshot_load(self, snap: torch.Tensor, state: "RLTState", row: int, M: torch.Tensor,
                      cache: torch.Tensor | None = None, T_max: int = 0) -> None:
        _check(lib().rlt_snapshot_load(self.handle, _ptr(snap), _ptr(state.buf), int(row), _ptr(cache), int(T_max),
                                       _ptr(M), M.shape[4], _stream()), "rlt_snapshot_load")

    def sample(self, logp: torch.Tensor, u: torch.Tensor, top_k: int = 0, top_p: float = 1.0,
               out: torch.Tensor | None = None, behaviour_logp: torch.Tensor | None = None) -> torch.Tensor:
        """rlt_sample: one token per row of logp [B, V] with the uniforms u [B]; `out` may be a
        column view of a token matrix (its stride is passed through).  A row without any probability
        gives token 0 with a log-probability of -inf and latches RLT_EDEVICE."""
        B = logp.shape[0]
        out = torch.empty(B, dtype=torch.int32, device=self.device) if out is None else out
        _check(lib().rlt_sample(self.handle, _ptr(logp), B, _ptr(u), int(top_k), float(top_p), _ptr(out),
                                out.stride(0), _ptr(behaviour_logp), _stream()), "rlt_sample")
        return out

    # ---------------------------------------------------------------- paged cache
    def alloc_pages(self, n_pages: int, page_size: int, n_kv_heads: int | None = None,
                    layers: int | None = None) -> torch.Tensor:
        """Pools of pages, [layers, n_pages, 2, n_kv_heads, page_size, head_dim] (defaults: the model's)."""
        c = self.cfg
        return torch.empty((c.L_E if layers is None else layers, n_pages, 2, n_kv_heads or c.n_heads, page_size,
                            c.head_dim), dtype=self.sdtype, device=self.device)

    def paged_batch(self, table: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor, N: int, max_q: int,
                    max_kv: int, page_size: int, n_kv_heads: int | None = None) -> PagedBatch:
        """Describe new tokens over a paged cache: table int32 [B, pages], q_start int32 [B + 1], kv_len
        int32 [B] (with the new tokens), N packed rows, and bounds of every sequence's new tokens and
        kv_len."""
        return PagedBatch(self, table, q_start, kv_len, N, max_q, max_kv, page_size,
                          self.cfg.n_heads if n_kv_heads is None else n_kv_heads)

    def _paged(self, batch: PagedBatch, pool: torch.Tensor):
        if batch.model is not self:
            raise ValueError("the batch was made for another model")
        return batch.args(pool)

    def paged_append(self, batch: PagedBatch, pool: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                     q: torch.Tensor | None = None, q_out: torch.Tensor | None = None) -> torch.Tensor | None:
        """rlt_paged_append: k, v [N, n_kv_heads, head_dim] (float32 or the model's dtype) into the pool
        [n_pages, 2, n_kv_heads, page_size, head_dim], the keys rotated; with q [N, n_heads, head_dim] the
        rotated queries are returned (in q_out)."""
        ref = self._paged(batch, pool)
        N, hd, dev, dt = batch.N, self.cfg.head_dim, self._dev, k.dtype
        if dt is not torch.float32 and dt is not self.sdtype:
            raise ValueError(f"k: need float32 or {self.sdtype}, got {dt}")
        shape = (N, batch.n_kv_heads, hd)
        kp, ks = _rows(k, "k", dt, dev, shape)
        vp, vs = _rows(v, "v", dt, dev, shape)
        H = qs = os = qp = op = 0
        if q is None:
            if q_out is not None:
                raise ValueError("q_out without q")
        else:
            H = q.shape[1]
            shape = (N, H, hd)
            qp, qs = _rows(q, "q", dt, dev, shape)
            if q_out is None:
                q_out = torch.empty(shape, dtype=self.sdtype, device=self.device)
            op, os = _rows(q_out, "q_out", self.sdtype, dev, shape)
        code = lib().rlt_paged_append(self.handle, ref, pool.data_ptr(), kp, ks, vp, vs, qp, qs, H, op, os,
                                      RLT_F32 if dt is torch.float32 else RLT_BF16, self._raw_stream())
        if code:
            raise RLTError(code, "rlt_paged_append")
        return q_out

    def paged_attention(self, batch: PagedBatch, pool: torch.Tensor, q: torch.Tensor, out: torch.Tensor | None = None,
                        scale: float = 0.0) -> torch.Tensor:
        """rlt_paged_attention: q [N, n_heads, head_dim] (rotated, the model's dtype) over the pool, which
        holds the new tokens already -> out, the same shape (rows behind the last sequence are left as
        they were).  scale 0: 1 / sqrt(head_dim)."""
        ref = self._paged(batch, pool)
        H, dev = q.shape[1], self._dev
        shape = (batch.N, H, self.cfg.head_dim)
        qp, qs = _rows(q, "q", self.sdtype, dev, shape)
        if out is None:
            out = torch.empty(shape, dtype=self.sdtype, device=self.device)
        op, os = _rows(out, "out", self.sdtype, dev, shape)
        # the workspace is the caller's stream's: from torch's allocator, for this call alone
        nb = batch.attention_workspace_bytes(H)
        ws = torch.empty(nb, dtype=torch.uint8, device=self.device) if nb else None
        code = lib().rlt_paged_attention(self.handle, ref, pool.data_ptr(), qp, qs, H, op, os, scale,
                                         None if ws is None else ws.data_ptr(), nb, self._raw_stream())
        if code:
            raise RLTError(code, "rlt_paged_attention")
        return out

    def encode_chunk(self, batch: PagedBatch, pools: torch.Tensor, tokens: torch.Tensor, e: torch.Tensor,
                     M: torch.Tensor) -> None:
        """rlt_encode_chunk: encode tokens int32 [N] over pools (alloc_pages); the new rows of e
        [B, T_alloc, d] and M [G, 2, B, n_heads, T_alloc, head_dim] are written in place."""
        c, dev = self.cfg, self._dev
        if pools.shape[0] != c.L_E or pools.dim() != 6 or not pools.is_contiguous():
            raise ValueError(f"pools: need {c.L_E} pools, contiguous, got {list(pools.shape)}")
        ref = self._paged(batch, pools[0])
        T_alloc = e.shape[1]
        _need(tokens, "tokens", torch.int32, dev, (batch.N,))
        _need(e, "e", self.sdtype, dev, (batch.B, T_alloc, c.d))
        _need(M, "M", self.sdtype, dev, (c.G, 2, batch.B, c.n_heads, T_alloc, c.head_dim))
        if not (tokens.is_contiguous() and e.is_contiguous() and M.is_contiguous()):
            raise ValueError("tokens, e and M must be contiguous")
        nb = lib().rlt_encode_chunk_workspace_bytes(self.handle, ref)
        ws = torch.empty(max(nb, 256), dtype=torch.uint8, device=self.device)
        _check(lib().rlt_encode_chunk(self.handle, ref, tokens.data_ptr(), pools.data_ptr(), e.data_ptr(), M.data_ptr(),
                                      T_alloc, ws.data_ptr(), nb, self._raw_stream()), "rlt_encode_chunk")

    # ---------------------------------------------------------------- logits before a draw
    def process_logits(self, logits: torch.Tensor, *, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                       bias: torch.Tensor | None = None, mask: torch.Tensor | None = None,
                       tokens: torch.Tensor | None = None, tok_len: torch.Tensor | None = None,
                       gen_start: torch.Tensor | None = None, repetition: torch.Tensor | None = None,
                       presence: torch.Tensor | None = None, frequency: torch.Tensor | None = None,
                       tau: torch.Tensor | None = None, out_lse: torch.Tensor | None = None) -> torch.Tensor:
        """rlt_process_logits: penalties over the history tokens int32 [B, n] (any strides; tok_len
        valid ones each, those from gen_start on generated), bias float32 [B or 1, V], mask int32
        [B or 1, ceil(V / 32)] of allowed bits, per-row float32 parameters; returns out, the
        log-probabilities that sample() draws from.  With lse, logits are log-probabilities at
        temperature 1.  out may be logits."""
        B, V, dev, f32 = logits.shape[0], self.cfg.V, self._dev, torch.float32
        _need(logits, "logits", f32, dev, (B, V))
        if out is None:
            out = torch.empty((B, V), dtype=f32, device=self.device)
        else:
            _need(out, "out", f32, dev, (B, V))
        xs, os = logits.stride(), out.stride()
        if xs[1] != 1 or os[1] != 1:
            raise ValueError("the rows of logits and out must be contiguous")
        a = LogitsArgs()
        a.x, a.x_stride = logits.data_ptr(), xs[0] if B > 1 else V
        a.out, a.out_stride = out.data_ptr(), os[0] if B > 1 else V
        if bias is not None:
            a.bias, a.bias_stride = self._broadcast_rows(bias, "bias", f32, B, V)
        if mask is not None:
            a.mask, a.mask_stride = self._broadcast_rows(mask, "mask", torch.int32, B, (V + 31) // 32)
        if tokens is not None:
            n = tokens.shape[1]
            _need(tokens, "tokens", torch.int32, dev, (B, n))
            a.tokens, a.n_tokens = tokens.data_ptr(), n
            a.seq_stride, a.tok_stride = tokens.stride()
            a.tok_len = self._row_vector(tok_len, "tok_len", torch.int32, B)
            a.gen_start = self._row_vector(gen_start, "gen_start", torch.int32, B)
        elif tok_len is not None or gen_start is not None:
            raise ValueError("tok_len and gen_start belong to tokens")
        a.lse = self._row_vector(lse, "lse", f32, B)
        a.repetition = self._row_vector(repetition, "repetition", f32, B)
        a.presence = self._row_vector(presence, "presence", f32, B)
        a.frequency = self._row_vector(frequency, "frequency", f32, B)
        a.tau = self._row_vector(tau, "tau", f32, B)
        a.out_lse = self._row_vector(out_lse, "out_lse", f32, B)
        code = lib().rlt_process_logits(self.handle, ctypes.byref(a), B, self._raw_stream())
        if code:
            raise RLTError(code, "rlt_process_logits")
        return out

    def _row_vector(self, t: torch.Tensor | None, what: str, dtype, B: int):
        if t is None:
            return None
        _need(t, what, dtype, self._dev, (B,))
        if B > 1 and t.stride(0) != 1:
            raise ValueError(f"{what}: must be contiguous")
        return t.data_ptr()

    def _broadcast_rows(self, t: torch.Tensor, what: str, dtype, B: int, n: int):
        """(address, row stride) of [B, n], or of [1, n] with a stride of 0."""
        rows = 1 if t.shape[0] == 1 else B
        _need(t, what, dtype, self._dev, (rows, n))
        if n > 1 and t.stride(1) != 1:
            raise ValueError(f"{what}: rows must be contiguous")
        return t.data_ptr(), t.stride(0) if rows > 1 else 0

    def generate(self, prompt: torch.Tensor, n_new: int, uniforms: torch.Tensor, tau: float = 1.0, top_k: int = 0,
                 top_p: float = 1.0, *, repetition=None, presence=None, frequency=None,
                 bias: torch.Tensor | None = None, mask=None):
        """Sample n_new tokens after each prompt row (all rows in lockstep): encode the prompt with a
        cache, step the decoder through it, then repeat [sample x_{t+1} from logp_t, encode it
        incrementally, step].  uniforms: float device [n_new, B].  Returns (tokens [B, P + n_new]
        int32, behaviour log-probs [B, n_new], prompt log-probs [B, P - 1] (entry t-1 = log p of
        x_{t+1}), the state after all P + n_new tokens).  Every step of the loop runs in the
        library's kernels; nothing but the error flag of a controlled call is copied to the host.

        With any of repetition, presence, frequency (numbers, or float32 device vectors [B]), bias
        (float32 [B or 1, V]) and mask (int32 [B or 1, ceil(V / 32)], or a function of the number of
        tokens generated so far and the tokens [B, t] that returns one) each draw is from the logits
        that process_logits makes of them: the prompt counts for repetition only.  What the device
        refused on the way, a row without an allowed token among it, is raised as RLTError at the end
        (of a captured call last_error() tells behind the replay)."""
        prompt = prompt.to(device=self.device, dtype=torch.int32).contiguous()
        B, P = prompt.shape
        T = P + n_new
        toks = torch.empty((T, B), dtype=torch.int32, device=self.device)     # row t = x_{t+1}
        toks[:P] = prompt.t()
        e, M, cache = self.encode_prefill(prompt, T_alloc=T, T_max=T)
        st = self.new_state(B)
        blp = torch.empty((n_new, B), dtype=torch.float32, device=self.device)
        lp_prompt = torch.zeros((max(P - 1, 0), B), dtype=torch.float32, device=self.device)
        row = torch.empty((B, self.cfg.V), dtype=torch.float32, device=self.device)
        control = None
        if any(x is not None for x in (repetition, presence, frequency, bias, mask)):
            def vector(x):
                return x if x is None or isinstance(x, torch.Tensor) else \
                    torch.full((B,), float(x), dtype=torch.float32, device=self.device)
            control = dict(repetition=vector(repetition), presence=vector(presence), frequency=vector(frequency),
                           tau=vector(tau), bias=bias, gen_start=torch.full((B,), P, dtype=torch.int32,
                                                                            device=self.device))
            lse = torch.empty(B, dtype=torch.float32, device=self.device)
        for t in range(1, T):                      # step t consumes x_t and predicts x_{t+1}
            if t < P:
                self.decode_step(st, e, M, next_tok=toks[t], tau=tau, logp_tok=lp_prompt[t - 1])
                continue
            if control is None:
                self.decode_step(st, e, M, tau=tau, logp_full=row)
            else:
                self.decode_step(st, e, M, tau=1.0, lse=lse, logp_full=row)
                allowed = mask(t - P, toks[:t].t()) if callable(mask) else mask
                self.process_logits(row, out=row, lse=lse, mask=allowed, tokens=toks[:t].t(), **control)
            self.sample(row, uniforms[t - P], top_k, top_p, out=toks[t], behaviour_logp=blp[t - P])
            self.encode_append(toks[t], t, cache, T, e, M)
        self.decode_step(st, e, M, tau=tau)         # the transition of x_T
        if control is not None and not torch.cuda.is_current_stream_capturing():
            self.check_device_errors()
        return toks.t().contiguous(), blp.t().contiguous(), lp_prompt.t().contiguous(), st

    # ---------------------------------------------------------------- decoder
    def new_state(self, B: int) -> RLTState:
        buf = torch.empty(lib().rlt_state_bytes(self.handle, B), dtype=torch.uint8, device=self.device)
        _check(lib().rlt_state_init(self.handle, _ptr(buf), B, _stream()), "rlt_state_init")
        return RLTState(self, B, buf)

    def reset_state(self, state: RLTState) -> RLTState:
        _check(lib().rlt_state_init(self.handle, _ptr(state.buf), state.B, _stream()), "rlt_state_init")
        return state

    def decode_step(self, state: RLTState, e: torch.Tensor, M: torch.Tensor, next_tok: torch.Tensor | None = None,
                    tau: float = 1.0, logp_tok: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    logp_full: torch.Tensor | None = None) -> None:
        """One transition H_{t-1} -> H_t in place; outputs go to the given device tensors."""
        B = state.B
        nb = lib().rlt_decode_workspace_bytes(self.handle, B)
        ws = self._workspace(("dec", B), nb)
        _check(lib().rlt_decode_step(self.handle, _ptr(state.buf), B, _ptr(e), _ptr(M), e.shape[1], _ptr(next_tok),
                                     float(tau), _ptr(logp_tok), _ptr(lse), _ptr(logp_full), _ptr(ws), ws.numel(),
                                     _stream()), "rlt_decode_step")

    def decode_step_noalloc(self, state: RLTState, e: torch.Tensor, M: torch.Tensor,
                            next_tok: torch.Tensor | None = None, tau: float = 1.0,
                            logp_tok: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                            logp_full: torch.Tensor | None = None) -> None:
        """rlt_decode_step without a caller workspace: the step's scratch is the library's static
        device array (see include/rlt.h for its size limit and the rules on overlapping calls)."""
        _check(lib().rlt_decode_step_noalloc(self.handle, _ptr(state.buf), state.B, _ptr(e), _ptr(M), e.shape[1],
                                             _ptr(next_tok), float(tau), _ptr(logp_tok), _ptr(lse), _ptr(logp_full),
                                             _stream()), "rlt_decode_step_noalloc")

    def replay(self, tokens: torch.Tensor, prompt_len, tau: float = 1.0, want_logp: bool = False,
               want_state: bool = False):
        """Exact current-policy replay; returns (score [B], logp_tok [B, T] | None, state | None)."""
        tokens = tokens.to(device=self.device, dtype=torch.int32).contiguous()
        B, T = tokens.shape
        P = torch.as_tensor(prompt_len, dtype=torch.int32).to(self.device).expand(B).contiguous()
        score = torch.empty(B, dtype=torch.float32, device=self.device)
        lp = torch.empty((B, T), dtype=torch.float32, device=self.device) if want_logp else None
        st = None
        if want_state:
            st = RLTState(self, B, torch.empty(lib().rlt_state_bytes(self.handle, B), dtype=torch.uint8,
                                               device=self.device))
        nb = lib().rlt_replay_workspace_bytes(self.handle, B, T)
        ws = self._workspace(("replay", B, T), nb)
        _check(lib().rlt_replay(self.handle, _ptr(tokens), B, T, _ptr(P), float(tau), _ptr(score), _ptr(lp),
                                _ptr(st.buf) if st else None, _ptr(ws), ws.numel(), _stream()), "rlt_replay")
        return score, lp, st

    def gemm_bf16(self, A: torch.Tensor, W: torch.Tensor, kernel: int = 0,
                  out: torch.Tensor | None = None) -> torch.Tensor:
        """C = A W^T (bf16 in, float32 out) with the kernel id of rlt_gemm_bf16 (0: the library's
        choice, 1: CUDA cores, 2 + v: row-tile variant v, 11 + s: few-row kernel, 16: weight
        streaming, 17: persistent, 18 + p: CTA-pair tiles 256 x (64 << p))."""
        A = A.to(self.device, torch.bfloat16).contiguous()
        W = W.to(self.device, torch.bfloat16).contiguous()
        M, K = A.shape
        N = W.shape[0]
        C = torch.empty((M, N), dtype=torch.float32, device=self.device) if out is None else out
        _check(lib().rlt_gemm_bf16(self.handle, _ptr(A), _ptr(W), _ptr(C), M, N, K, kernel, _stream()),
               "rlt_gemm_bf16")
        return C

    def selftest_wait_timeout(self, A: torch.Tensor, W: torch.Tensor, C: torch.Tensor, kernel: int,
                              wait_ns: int) -> None:
        """Launch tensor-core kernel `kernel` in its no-load self-test mode (every wait bounded by
        wait_ns); the next last_error() reports RLT_ETIMEOUT."""
        M, K = A.shape
        N = W.shape[0]
        _check(lib().rlt_selftest_wait_timeout(self.handle, _ptr(A), _ptr(W), _ptr(C), M, N, K, kernel,
                                               int(wait_ns), _stream()), "rlt_selftest_wait_timeout")

    def profile_start(self, kinds=None) -> None:
        """Bracket every launch of the given kernel kinds (names of KERNEL_KINDS) with CUDA events."""
        kinds = KERNEL_KINDS if kinds is None else kinds
        mask = 0
        for k in kinds:
            mask |= 1 << KERNEL_KINDS.index(k)
        _check(lib().rlt_profile_start(self.handle, mask), "rlt_profile_start")

    def profile_stop(self) -> dict:
        """Per kind: (summed milliseconds, bracketed launches)."""
        n = len(KERNEL_KINDS)
        ms = (ctypes.c_double * n)()
        cnt = (ctypes.c_uint64 * n)()
        _check(lib().rlt_profile_stop(self.handle, ms, cnt), "rlt_profile_stop")
        return {k: (ms[i], cnt[i]) for i, k in enumerate(KERNEL_KINDS) if cnt[i]}

    def last_error(self) -> int:
        return lib().rlt_last_error(self.handle, _stream())

    def check_device_errors(self) -> None:
        _check(self.last_error(), "device-side check")
