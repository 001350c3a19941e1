"""ctypes binding of libepget (include/ep_get.h): argument marshalling only.

Every step of the path runs in the library's HIP kernels; this module turns
tensors into raw device pointers, fills the ``ep_problem`` struct, passes the
current HIP stream and raises on error codes.  Loading fails loudly if the
library has not been built.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libepget.so")

EP_OK = 0
EP_ERR_INVALID_ARG = -1
EP_ERR_HIP = -2
EP_ERR_CAPACITY = -3
EP_ERR_BAD_EXPERT = -4
EP_ERR_SCRATCH_LIMIT = -5
EP_NOALLOC_SCRATCH_BYTES = 8 << 20

EP_MAX_RANKS = 1024
EP_MAX_EXPERTS = 2048
EP_MAX_EXPERTS_PER_RANK = 256
EP_MAX_TOPK = 32
EP_MAX_HIDDEN = 1 << 24
EP_MAX_FEATURES = 1 << 16
EP_MOE_TOKENS_MAX = 128

EP_ACT_NONE = 0
EP_ACT_RELU = 1
EP_ACT_GELU = 2
EP_ACT_SILU = 3
EP_ACT_SWIGLU = 4
EP_ACT_GEGLU = 5

EP_WEIGHTS_BF16 = 0
EP_WEIGHTS_FP8 = 1
EP_WEIGHTS_FP4 = 2

EP_SCORE_SOFTMAX = 0
EP_SCORE_SIGMOID = 1

EP_GRAD_BF16 = 0
EP_GRAD_FP32 = 1

# Every function the C header declares, checked by the test-suite.
EXPORTS = ("ep_workspace_bytes", "ep_rank_stride_hint", "ep_get_layout", "ep_dispatch",
           "ep_layout_dispatch", "ep_combine", "ep_quantize_fp8", "ep_dispatch_fp8",
           "ep_layout_dispatch_fp8", "ep_get_group_layout", "ep_dispatch_hier", "ep_combine_hier",
           "ep_combine_topk_weights", "ep_read_status", "ep_error_string",
           "ep_layout_dispatch_noalloc", "ep_combine_backward", "ep_expert_product",
           "ep_expert_product_fp8", "ep_product_workspace_bytes", "ep_expert_product_backward",
           "ep_moe_tokens_workspace_bytes", "ep_moe_tokens", "ep_moe_tokens_fp8",
           "ep_expert_product_fp4", "ep_moe_tokens_fp4", "ep_route_workspace_bytes", "ep_route",
           "ep_balance_loss", "ep_route_backward", "ep_grad_workspace_bytes", "ep_grad_square_sum",
           "ep_grad_clip", "ep_moe_tokens_weights_workspace_bytes")


class EpError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {error_string(code)} ({code})")


class Problem(ctypes.Structure):
    """``ep_problem``: T, H, E, K, R, G, A and the rank slice stride S."""
    _fields_ = [
        ("num_tokens", ctypes.c_int32),
        ("hidden", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("num_topk", ctypes.c_int32),
        ("num_ranks", ctypes.c_int32),
        ("num_groups", ctypes.c_int32),
        ("expert_alignment", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("rank_stride_rows", ctypes.c_int64),
    ]

    @classmethod
    def make(cls, T, H, E, K, R, G=1, A=1, S=0):
        return cls(T, H, E, K, R, G, A, 0, S)

    @property
    def num_rows(self) -> int:
        return self.num_ranks * self.rank_stride_rows


class Product(ctypes.Structure):
    """``ep_product``: inputs C, outputs N and the activation of the experts' products."""
    _fields_ = [
        ("in_features", ctypes.c_int32),
        ("out_features", ctypes.c_int32),
        ("activation", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]

    @classmethod
    def make(cls, C, N, activation=EP_ACT_NONE):
        return cls(C, N, activation, 0)

    @property
    def weight_rows(self) -> int:
        """M: rows of an expert's weight, both halves of a gated activation."""
        return self.out_features * (2 if self.activation in (EP_ACT_SWIGLU, EP_ACT_GEGLU) else 1)


class Router(ctypes.Structure):
    """``ep_router``: scores, normalisation, the logits' type and the factor of the weights."""
    _fields_ = [
        ("score", ctypes.c_int32),
        ("normalise", ctypes.c_int32),
        ("logits_bf16", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]

    @classmethod
    def make(cls, score=EP_SCORE_SOFTMAX, normalise=True, scale=1.0, logits_bf16=False):
        return cls(score, int(normalise), int(logits_bf16), scale)


class Grad(ctypes.Structure):
    """``ep_grad``: one gradient, and where ep_grad_clip writes it."""
    _fields_ = [
        ("grad", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("count", ctypes.c_int64),
        ("type", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class Grads:
    """The gradients of ep_grad_square_sum and ep_grad_clip, as the host array of ``ep_grad`` that the calls take.
    It keeps the tensors, whose addresses it holds."""

    def __init__(self, array, tensors):
        self.array, self.tensors = array, tensors

    def __len__(self) -> int:
        return len(self.array)

    @classmethod
    def make(cls, grads, outs=None):
        """Of bf16 and fp32 tensors, clipped in place unless `outs` names other ones of the same types and sizes."""
        import torch

        grads = list(grads)
        outs = grads if outs is None else list(outs)
        if len(outs) != len(grads):
            raise ValueError(f"outs: {len(outs)} tensors for {len(grads)} gradients")
        if len({t.device for t in (*grads, *outs)}) > 1:
            raise ValueError("gradients on more than one device: a list, and a sum, for each")
        first = {}  # a gradient that is clipped twice at once has no defined result
        for i, o in enumerate(outs):
            if o.numel() and first.setdefault(o.data_ptr(), i) != i:
                raise ValueError(f"outs: tensors {first[o.data_ptr()]} and {i} are the same memory")
        types = {torch.bfloat16: (EP_GRAD_BF16, "bf16"), torch.float32: (EP_GRAD_FP32, "float")}
        array = (Grad * len(grads))()
        for i, (g, o) in enumerate(zip(grads, outs)):
            if g.dtype not in types or o.dtype != g.dtype:
                raise ValueError(f"gradient {i}: dtype {g.dtype} into {o.dtype}, expected bfloat16 or float32 in both")
            if o.numel() != g.numel():
                raise ValueError(f"outs: tensor {i} has {o.numel()} elements, its gradient {g.numel()}")
            code, name = types[g.dtype]
            array[i] = Grad(_arg(g, f"gradient {i}", name, g.numel()), _arg(o, f"out {i}", name, g.numel()), g.numel(), code, 0)
        return cls(array, (grads, outs))


_lib = None


def load():
    """Load libepget.so (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                              "or python -m combine_ep_get_amd.build")
        lib = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(Problem)
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        lib.ep_workspace_bytes.restype = sz
        lib.ep_workspace_bytes.argtypes = [P]
        lib.ep_rank_stride_hint.restype = ctypes.c_int64
        lib.ep_rank_stride_hint.argtypes = [P]
        lib.ep_get_layout.restype = ctypes.c_int
        lib.ep_get_layout.argtypes = [P] + [vp] * 10 + [sz, vp]
        lib.ep_dispatch.restype = ctypes.c_int
        lib.ep_dispatch.argtypes = [P] + [vp] * 6 + [vp]
        lib.ep_layout_dispatch.restype = ctypes.c_int
        lib.ep_layout_dispatch.argtypes = [P] + [vp] * 10 + [sz] + [vp] * 5 + [vp]
        lib.ep_layout_dispatch_noalloc.restype = ctypes.c_int
        lib.ep_layout_dispatch_noalloc.argtypes = [P] + [vp] * 10 + [vp] * 5 + [vp]
        lib.ep_combine.restype = ctypes.c_int
        lib.ep_combine.argtypes = [P] + [vp] * 4 + [vp]
        lib.ep_quantize_fp8.restype = ctypes.c_int
        lib.ep_quantize_fp8.argtypes = [P] + [vp] * 3 + [vp]
        lib.ep_dispatch_fp8.restype = ctypes.c_int
        lib.ep_dispatch_fp8.argtypes = [P] + [vp] * 6 + [ctypes.c_int64, ctypes.c_int64] + [vp] * 2 + [vp]
        i64 = ctypes.c_int64
        lib.ep_layout_dispatch_fp8.restype = ctypes.c_int
        lib.ep_layout_dispatch_fp8.argtypes = [P] + [vp] * 10 + [sz] + [vp] * 5 + [i64, i64] + [vp] * 2 + [vp]
        lib.ep_get_group_layout.restype = ctypes.c_int
        lib.ep_get_group_layout.argtypes = [P, vp, i64, vp, vp, vp]
        lib.ep_dispatch_hier.restype = ctypes.c_int
        lib.ep_dispatch_hier.argtypes = [P, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp]
        lib.ep_combine_hier.restype = ctypes.c_int
        lib.ep_combine_hier.argtypes = [P, vp, vp, vp, vp, i64, vp, vp, vp]
        lib.ep_combine_topk_weights.restype = ctypes.c_int
        lib.ep_combine_topk_weights.argtypes = [P] + [vp] * 3 + [vp]
        Q = ctypes.POINTER(Product)
        lib.ep_combine_backward.restype = ctypes.c_int
        lib.ep_combine_backward.argtypes = [P] + [vp] * 6 + [vp]
        lib.ep_expert_product.restype = ctypes.c_int
        lib.ep_expert_product.argtypes = [P, Q] + [vp] * 8 + [vp]
        lib.ep_expert_product_fp8.restype = ctypes.c_int
        lib.ep_expert_product_fp8.argtypes = [P, Q] + [vp] * 2 + [i64, i64] + [vp] * 7 + [vp]
        lib.ep_product_workspace_bytes.restype = sz
        lib.ep_product_workspace_bytes.argtypes = [P, Q]
        lib.ep_expert_product_backward.restype = ctypes.c_int
        lib.ep_expert_product_backward.argtypes = [P, Q] + [vp] * 12 + [sz, vp]
        lib.ep_moe_tokens_workspace_bytes.restype = sz
        lib.ep_moe_tokens_workspace_bytes.argtypes = [P, Q]
        lib.ep_moe_tokens_weights_workspace_bytes.restype = sz
        lib.ep_moe_tokens_weights_workspace_bytes.argtypes = [P, Q, ctypes.c_int32]
        lib.ep_moe_tokens.restype = ctypes.c_int
        lib.ep_moe_tokens.argtypes = [P, Q] + [vp] * 10 + [sz, vp]
        lib.ep_moe_tokens_fp8.restype = ctypes.c_int
        lib.ep_moe_tokens_fp8.argtypes = [P, Q] + [vp] * 12 + [sz, vp]
        lib.ep_expert_product_fp4.restype = ctypes.c_int
        lib.ep_expert_product_fp4.argtypes = [P, Q] + [vp] * 8 + [vp]
        lib.ep_moe_tokens_fp4.restype = ctypes.c_int
        lib.ep_moe_tokens_fp4.argtypes = [P, Q] + [vp] * 12 + [sz, vp]
        RT = ctypes.POINTER(Router)
        lib.ep_route_workspace_bytes.restype = sz
        lib.ep_route_workspace_bytes.argtypes = [P, RT]
        lib.ep_route.restype = ctypes.c_int
        lib.ep_route.argtypes = [P, RT] + [vp] * 10 + [sz, vp]
        lib.ep_balance_loss.restype = ctypes.c_int
        lib.ep_balance_loss.argtypes = [P, RT] + [vp] * 8 + [sz, vp]
        lib.ep_route_backward.restype = ctypes.c_int
        lib.ep_route_backward.argtypes = [P, RT] + [vp] * 8 + [vp]
        lib.ep_grad_workspace_bytes.restype = sz
        lib.ep_grad_workspace_bytes.argtypes = [vp, ctypes.c_int32]
        lib.ep_grad_square_sum.restype = ctypes.c_int
        lib.ep_grad_square_sum.argtypes = [vp, ctypes.c_int32, vp, vp, sz, vp]
        lib.ep_grad_clip.restype = ctypes.c_int
        lib.ep_grad_clip.argtypes = [vp, ctypes.c_int32, vp, ctypes.c_float, vp, vp]
        lib.ep_read_status.restype = ctypes.c_int
        lib.ep_read_status.argtypes = [vp, vp]
        lib.ep_error_string.restype = ctypes.c_char_p
        lib.ep_error_string.argtypes = [ctypes.c_int]
        _lib = lib
    return _lib


# Element types the C calls read, by the C type of the argument (filled on
# first use, so that importing the package does not import torch).
_DTYPES: dict = {}


def _dtypes():
    if not _DTYPES:
        import torch

        def with_named(types, name):  # a type that not every torch has
            t = getattr(torch, name, None)
            return types if t is None else (*types, t)

        _DTYPES.update({
            "int32": (torch.int32,),
            "int64": (torch.int64,),
            "double": (torch.float64,),
            "e2m1": with_named((torch.uint8, torch.int8), "float4_e2m1fn_x2"),  # two codes a byte
            "e8m0": with_named((torch.uint8, torch.int8), "float8_e8m0fnu"),
            "float": (torch.float32,),
            "uint8": (torch.uint8, torch.bool),
            "bf16": (torch.bfloat16, torch.int16, torch.uint16),
            "e4m3": (torch.float8_e4m3fn, torch.uint8, torch.int8),
            "bytes": None,
        })
    return _DTYPES


def _arg(t, what: str, ctype: str, count: int):
    """Pointer for argument `what` of C element type `ctype`, which the call
    reads or writes over `count` elements.  None gives NULL; an int is taken
    as a raw device address, unchecked.  A tensor must be dense, of that
    element type, hold at least `count` elements (bytes for "bytes") and be
    on the GPU: the kernels would read past a short array, and a host
    address in a kernel is a GPU memory fault."""
    if t is None or isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError(f"{what}: libepget takes contiguous arrays; call .contiguous() first")
    allowed = (_DTYPES or _dtypes())[ctype]
    if allowed is not None and t.dtype not in allowed:
        raise ValueError(f"{what}: dtype {t.dtype}, expected one of {allowed}")
    have = t.numel() * t.element_size() if allowed is None else t.numel()
    if have < count:
        raise ValueError(f"{what}: {have} {'bytes' if allowed is None else 'elements'}, "
                         f"the call uses {count}")
    if not t.is_cuda:
        raise ValueError(f"{what}: a {t.device.type} tensor; the library takes device memory")
    return t.data_ptr()


def _sizes(problem):
    """T, H, K, E, R, G and the receive rows R * S of a problem."""
    return (problem.num_tokens, problem.hidden, problem.num_topk, problem.num_experts,
            problem.num_ranks, problem.num_groups, problem.num_ranks * problem.rank_stride_rows)


def _layout_ptrs(problem, topk_idx, expert_count, expert_offset, rank_row_count, rank_token_count,
                 group_token_count, is_token_in_rank, token_slot, cumulative_expert_recv,
                 workspace, workspace_bytes):
    T, _, K, E, R, G, _ = _sizes(problem)
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    return (_arg(topk_idx, "topk_idx", "int32", T * K), _arg(expert_count, "expert_count", "int32", E),
            _arg(expert_offset, "expert_offset", "int32", E),
            _arg(rank_row_count, "rank_row_count", "int32", R),
            _arg(rank_token_count, "rank_token_count", "int32", R),
            _arg(group_token_count, "group_token_count", "int32", G),
            _arg(is_token_in_rank, "is_token_in_rank", "uint8", T * R),
            _arg(token_slot, "token_slot", "int32", T * K),
            _arg(cumulative_expert_recv, "cumulative_expert_recv", "int64", E),
            _arg(workspace, "workspace", "bytes", workspace_bytes), workspace_bytes)


def _fp8_rows_ptrs(problem, x_fp8, x_sf, recv_x_fp8, recv_sf, sf_token_stride, sf_hidden_stride):
    T, H, _, _, _, _, rows = _sizes(problem)
    nsf = H // 128
    sf_span = (rows - 1) * sf_token_stride + (nsf - 1) * sf_hidden_stride + 1 if rows and nsf else 0
    return (_arg(x_fp8, "x_fp8", "e4m3", T * H), _arg(x_sf, "x_sf", "float", T * nsf),
            _arg(recv_x_fp8, "recv_x_fp8", "e4m3", rows * H), _arg(recv_sf, "recv_sf", "float", sf_span))


def _stream(stream):
    if stream is None:
        # the raw handle where torch has it (a private name): the public call
        # builds an object around it, which takes as long as the launch (2.9 us
        # against 0.4)
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _on_current_device(stream, *tensors) -> None:
    """The calls run on the current device, unless the caller names a stream: refuses tensors of another one.  (Those of
    the host are _arg's to refuse.)"""
    if stream is not None:
        return
    here = None
    for t in tensors:
        if t is None or isinstance(t, int):
            continue
        device = t.get_device()
        if device != here and device >= 0:
            if here is None:
                import torch
                here = torch.cuda.current_device()
            if device != here:
                raise ValueError(f"a tensor on device {device} with device {here} current; "
                                 "use torch.cuda.device(...) around the call")


def error_string(code: int) -> str:
    return load().ep_error_string(code).decode()


def _check(rc: int, where: str) -> int:
    if rc != EP_OK:
        raise EpError(rc, where)
    return rc


class BoundCall:
    """One entry point with its arguments marshalled once.  Calling it issues
    the same C call again (same pointers, sizes and stream), so a loop that
    repeats a step pays only for the call itself.  The tensors must stay
    alive and in place while it is used.  The problem is copied when the
    call is bound: the tensors were checked against its sizes then, so later
    changes to the caller's struct are not seen (bind again instead)."""

    def __init__(self, name: str, problem: Problem, args: tuple):
        self.name = name
        self._fn = getattr(load(), name)
        self.problem = Problem.from_buffer_copy(problem)
        self._args = (ctypes.byref(self.problem), *args)

    def __call__(self) -> int:
        return _check(self._fn(*self._args), self.name)


def _run(name: str, problem: Problem, args: tuple, bind: bool):
    """Calls the entry point on `problem` and args now, or with bind=True
    returns it as a BoundCall."""
    if bind:
        return BoundCall(name, problem, args)
    return _check(getattr(load(), name)(ctypes.byref(problem), *args), name)


def ep_workspace_bytes(problem: Problem) -> int:
    return load().ep_workspace_bytes(ctypes.byref(problem))


def ep_rank_stride_hint(problem: Problem) -> int:
    return load().ep_rank_stride_hint(ctypes.byref(problem))


def ep_get_layout(problem, topk_idx, expert_count, expert_offset, rank_row_count,
                  rank_token_count, group_token_count, is_token_in_rank, token_slot,
                  cumulative_expert_recv, workspace, workspace_bytes=None, stream=None, bind=False):
    lay = _layout_ptrs(problem, topk_idx, expert_count, expert_offset, rank_row_count,
                       rank_token_count, group_token_count, is_token_in_rank, token_slot,
                       cumulative_expert_recv, workspace, workspace_bytes)
    return _run("ep_get_layout", problem, (*lay, _stream(stream)), bind)


def _dispatch_ptrs(problem, x, topk_weights, recv_x, recv_src_token, recv_weight):
    T, H, K, _, _, _, rows = _sizes(problem)
    return (_arg(x, "x", "bf16", T * H), _arg(topk_weights, "topk_weights", "float", T * K),
            _arg(recv_x, "recv_x", "bf16", rows * H), _arg(recv_src_token, "recv_src_token", "int32", rows),
            _arg(recv_weight, "recv_weight", "float", rows))


def ep_dispatch(problem, x, topk_weights, token_slot, recv_x, recv_src_token=None,
                recv_weight=None, stream=None, bind=False):
    T, _, K, _, _, _, _ = _sizes(problem)
    px, pw, prx, psrc, prw = _dispatch_ptrs(problem, x, topk_weights, recv_x, recv_src_token, recv_weight)
    return _run("ep_dispatch", problem, (px, pw, _arg(token_slot, "token_slot", "int32", T * K),
        prx, psrc, prw, _stream(stream)), bind)


def ep_layout_dispatch(problem, topk_idx, expert_count, expert_offset, rank_row_count,
                       rank_token_count, group_token_count, is_token_in_rank, token_slot,
                       cumulative_expert_recv, workspace, workspace_bytes, x, topk_weights, recv_x,
                       recv_src_token=None, recv_weight=None, stream=None, bind=False):
    """ep_get_layout followed by ep_dispatch (one kernel for decode-sized batches)."""
    lay = _layout_ptrs(problem, topk_idx, expert_count, expert_offset, rank_row_count,
                       rank_token_count, group_token_count, is_token_in_rank, token_slot,
                       cumulative_expert_recv, workspace, workspace_bytes)
    rows = _dispatch_ptrs(problem, x, topk_weights, recv_x, recv_src_token, recv_weight)
    return _run("ep_layout_dispatch", problem, (*lay, *rows, _stream(stream)), bind)


def ep_layout_dispatch_noalloc(problem, topk_idx, expert_count, expert_offset, rank_row_count,
                               rank_token_count, group_token_count, is_token_in_rank, token_slot,
                               cumulative_expert_recv, status, x, topk_weights, recv_x,
                               recv_src_token=None, recv_weight=None, stream=None, bind=False):
    """ep_layout_dispatch with the layout scratch in the library's static
    device buffer (no workspace argument); the status word goes to `status`
    (one int32 on the device, read with ep_read_status)."""
    T, _, K, E, R, G, _ = _sizes(problem)
    lay = (_arg(topk_idx, "topk_idx", "int32", T * K), _arg(expert_count, "expert_count", "int32", E),
           _arg(expert_offset, "expert_offset", "int32", E),
           _arg(rank_row_count, "rank_row_count", "int32", R),
           _arg(rank_token_count, "rank_token_count", "int32", R),
           _arg(group_token_count, "group_token_count", "int32", G),
           _arg(is_token_in_rank, "is_token_in_rank", "uint8", T * R),
           _arg(token_slot, "token_slot", "int32", T * K),
           _arg(cumulative_expert_recv, "cumulative_expert_recv", "int64", E),
           _arg(status, "status", "int32", 1))
    rows = _dispatch_ptrs(problem, x, topk_weights, recv_x, recv_src_token, recv_weight)
    return _run("ep_layout_dispatch_noalloc", problem, (*lay, *rows, _stream(stream)), bind)


def ep_combine(problem, y, token_slot, topk_weights, out, stream=None, bind=False):
    T, H, K, _, _, _, rows = _sizes(problem)
    return _run("ep_combine", problem, (_arg(y, "y", "bf16", rows * H),
        _arg(token_slot, "token_slot", "int32", T * K),
        _arg(topk_weights, "topk_weights", "float", T * K),
        _arg(out, "out", "bf16", T * H), _stream(stream)), bind)


def ep_quantize_fp8(problem, x, x_fp8, x_sf, stream=None, bind=False):
    T, H, _, _, _, _, _ = _sizes(problem)
    return _run("ep_quantize_fp8", problem, (_arg(x, "x", "bf16", T * H),
        _arg(x_fp8, "x_fp8", "e4m3", T * H),
        _arg(x_sf, "x_sf", "float", T * (H // 128)), _stream(stream)), bind)


def ep_dispatch_fp8(problem, x_fp8, x_sf, topk_weights, token_slot, recv_x_fp8, recv_sf,
                    sf_token_stride, sf_hidden_stride, recv_src_token=None, recv_weight=None,
                    stream=None, bind=False):
    T, _, K, _, _, _, rows = _sizes(problem)
    px, psf, prx, prsf = _fp8_rows_ptrs(problem, x_fp8, x_sf, recv_x_fp8, recv_sf, sf_token_stride,
                                        sf_hidden_stride)
    return _run("ep_dispatch_fp8", problem, (px, psf,
        _arg(topk_weights, "topk_weights", "float", T * K),
        _arg(token_slot, "token_slot", "int32", T * K), prx, prsf,
        sf_token_stride, sf_hidden_stride,
        _arg(recv_src_token, "recv_src_token", "int32", rows),
        _arg(recv_weight, "recv_weight", "float", rows), _stream(stream)), bind)


def ep_layout_dispatch_fp8(problem, topk_idx, expert_count, expert_offset, rank_row_count,
                           rank_token_count, group_token_count, is_token_in_rank, token_slot,
                           cumulative_expert_recv, workspace, workspace_bytes, x_fp8, x_sf,
                           topk_weights, recv_x_fp8, recv_sf, sf_token_stride, sf_hidden_stride,
                           recv_src_token=None, recv_weight=None, stream=None, bind=False):
    """ep_get_layout followed by ep_dispatch_fp8 (one kernel for decode-sized batches)."""
    T, _, K, _, _, _, rows = _sizes(problem)
    lay = _layout_ptrs(problem, topk_idx, expert_count, expert_offset, rank_row_count,
                       rank_token_count, group_token_count, is_token_in_rank, token_slot,
                       cumulative_expert_recv, workspace, workspace_bytes)
    px, psf, prx, prsf = _fp8_rows_ptrs(problem, x_fp8, x_sf, recv_x_fp8, recv_sf, sf_token_stride,
                                        sf_hidden_stride)
    return _run("ep_layout_dispatch_fp8", problem, (*lay, px, psf,
        _arg(topk_weights, "topk_weights", "float", T * K), prx, prsf,
        sf_token_stride, sf_hidden_stride,
        _arg(recv_src_token, "recv_src_token", "int32", rows),
        _arg(recv_weight, "recv_weight", "float", rows),
        _stream(stream)), bind)


def ep_get_group_layout(problem, is_token_in_rank, group_stride_rows, group_slot, status=None,
                        stream=None, bind=False):
    """Group slots of the two-level path; `status` (one int32 on the device,
    e.g. the layout's workspace) is lowered to EP_ERR_CAPACITY when a group
    overflows SG rows."""
    T, _, _, _, R, G, _ = _sizes(problem)
    return _run("ep_get_group_layout", problem, (
        _arg(is_token_in_rank, "is_token_in_rank", "uint8", T * R),
        group_stride_rows, _arg(group_slot, "group_slot", "int32", T * G),
        _arg(status, "status", "bytes", 4), _stream(stream)), bind)


def ep_dispatch_hier(problem, x, topk_weights, token_slot, group_slot, group_stride_rows,
                     group_buf, recv_x, recv_src_token=None, recv_weight=None, stream=None, bind=False):
    T, H, K, _, _, G, _ = _sizes(problem)
    px, pw, prx, psrc, prw = _dispatch_ptrs(problem, x, topk_weights, recv_x, recv_src_token, recv_weight)
    return _run("ep_dispatch_hier", problem, (px, pw,
        _arg(token_slot, "token_slot", "int32", T * K),
        _arg(group_slot, "group_slot", "int32", T * G), group_stride_rows,
        _arg(group_buf, "group_buf", "bf16", G * group_stride_rows * H),
        prx, psrc, prw, _stream(stream)), bind)


def ep_combine_hier(problem, y, token_slot, topk_weights, group_slot, group_stride_rows,
                    group_buf, out, stream=None, bind=False):
    T, H, K, _, _, G, rows = _sizes(problem)
    return _run("ep_combine_hier", problem, (_arg(y, "y", "bf16", rows * H),
        _arg(token_slot, "token_slot", "int32", T * K),
        _arg(topk_weights, "topk_weights", "float", T * K),
        _arg(group_slot, "group_slot", "int32", T * G), group_stride_rows,
        _arg(group_buf, "group_buf", "bf16", G * group_stride_rows * H),
        _arg(out, "out", "bf16", T * H), _stream(stream)), bind)


def ep_combine_topk_weights(problem, recv_weight, token_slot, combined_topk_weights,
                            stream=None, bind=False):
    T, _, K, _, _, _, rows = _sizes(problem)
    return _run("ep_combine_topk_weights", problem, (
        _arg(recv_weight, "recv_weight", "float", rows),
        _arg(token_slot, "token_slot", "int32", T * K),
        _arg(combined_topk_weights, "combined_topk_weights", "float",
        T * K), _stream(stream)), bind)


def ep_combine_backward(problem, dout, y, token_slot, topk_weights, dy=None, dweights=None, stream=None,
                        bind=False):
    """Gradient of ep_combine: dy (which may be y) and the top-k weights' gradients."""
    T, H, K, _, _, _, rows = _sizes(problem)
    return _run("ep_combine_backward", problem, (_arg(dout, "dout", "bf16", T * H),
        _arg(y, "y", "bf16", rows * H), _arg(token_slot, "token_slot", "int32", T * K),
        _arg(topk_weights, "topk_weights", "float", T * K), _arg(dy, "dy", "bf16", rows * H),
        _arg(dweights, "dweights", "float", T * K), _stream(stream)), bind)


def _product_sizes(problem, product, expert_count):
    """E, C, N, M and the rows of x and out: the receive buffer's, or T for a
    dense product (no expert arrays)."""
    rows = problem.num_ranks * problem.rank_stride_rows if expert_count is not None else problem.num_tokens
    return problem.num_experts, product.in_features, product.out_features, product.weight_rows, rows


def _product_ref(product, bind):
    """The product (or router) by reference; a bound call keeps a copy of its own."""
    return ctypes.byref(type(product).from_buffer_copy(product) if bind else product)


def ep_expert_product(problem, product, x, expert_count, expert_offset, weight, bias=None, residual=None, pre=None,
                      out=None, stream=None, bind=False):
    """out = act(x W[e]^T + bias[e]) + residual on the experts' rows; `pre`
    takes the pre-activations that the backward call reads."""
    E, C, N, M, rows = _product_sizes(problem, product, expert_count)
    return _run("ep_expert_product", problem, (_product_ref(product, bind), _arg(x, "x", "bf16", rows * C),
        _arg(expert_count, "expert_count", "int32", E), _arg(expert_offset, "expert_offset", "int32", E),
        _arg(weight, "weight", "bf16", E * M * C), _arg(bias, "bias", "float", E * M),
        _arg(residual, "residual", "bf16", rows * N), _arg(pre, "pre", "bf16", rows * M),
        _arg(out, "out", "bf16", rows * N), _stream(stream)), bind)


def ep_expert_product_fp8(problem, product, x_fp8, x_sf, sf_token_stride, sf_hidden_stride, expert_count,
                          expert_offset, w_fp8, w_sf, bias=None, residual=None, out=None, stream=None, bind=False):
    """ep_expert_product on e4m3 rows and weights with fp32 scales."""
    E, C, N, M, rows = _product_sizes(problem, product, expert_count)
    nsf = C // 128
    span = (rows - 1) * sf_token_stride + (nsf - 1) * sf_hidden_stride + 1 if rows and nsf else 0
    return _run("ep_expert_product_fp8", problem, (_product_ref(product, bind), _arg(x_fp8, "x_fp8", "e4m3", rows * C),
        _arg(x_sf, "x_sf", "float", span), sf_token_stride, sf_hidden_stride,
        _arg(expert_count, "expert_count", "int32", E), _arg(expert_offset, "expert_offset", "int32", E),
        _arg(w_fp8, "w_fp8", "e4m3", E * M * C), _arg(w_sf, "w_sf", "float", E * (M // 128) * nsf),
        _arg(bias, "bias", "float", E * M), _arg(residual, "residual", "bf16", rows * N),
        _arg(out, "out", "bf16", rows * N), _stream(stream)), bind)


def ep_product_workspace_bytes(problem: Problem, product: Product) -> int:
    return load().ep_product_workspace_bytes(ctypes.byref(problem), ctypes.byref(product))


def ep_expert_product_backward(problem, product, dout, pre, x, expert_count, expert_offset, weight, dpre=None, dx=None,
                               dweight=None, dweight_acc=None, dbias=None, workspace=None, workspace_bytes=None,
                               stream=None, bind=False):
    """Gradients of ep_expert_product: dpre, dx, dweight (bf16) or dweight_acc
    (fp32, added to), dbias; those that are None are not computed."""
    E, C, N, M, rows = _product_sizes(problem, product, expert_count)
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return _run("ep_expert_product_backward", problem, (_product_ref(product, bind),
        _arg(dout, "dout", "bf16", rows * N), _arg(pre, "pre", "bf16", rows * M), _arg(x, "x", "bf16", rows * C),
        _arg(expert_count, "expert_count", "int32", E), _arg(expert_offset, "expert_offset", "int32", E),
        _arg(weight, "weight", "bf16", E * M * C), _arg(dpre, "dpre", "bf16", rows * M),
        _arg(dx, "dx", "bf16", rows * C), _arg(dweight, "dweight", "bf16", E * M * C),
        _arg(dweight_acc, "dweight_acc", "float", E * M * C), _arg(dbias, "dbias", "float", E * M),
        _arg(workspace, "workspace", "bytes", workspace_bytes), workspace_bytes, _stream(stream)), bind)


def ep_moe_tokens_workspace_bytes(problem: Problem, product: Product) -> int:
    """Bytes that serve each of the ep_moe_tokens calls of these sizes."""
    return load().ep_moe_tokens_workspace_bytes(ctypes.byref(problem), ctypes.byref(product))


def ep_moe_tokens_weights_workspace_bytes(problem: Problem, product: Product, weights: int) -> int:
    """Bytes that the call on these weights (EP_WEIGHTS_*) needs; 0 if it refuses the sizes."""
    return load().ep_moe_tokens_weights_workspace_bytes(ctypes.byref(problem), ctypes.byref(product), weights)


def _tokens_ptrs(problem, product, x, topk_idx, topk_weights, w1, w1_sf, b1, w2, w2_sf, b2, residual, out, workspace,
                 workspace_bytes, wtype, stream, bind):
    T, H, K, E, _, _, _ = _sizes(problem)
    I, M = product.out_features, product.weight_rows
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    codes = 2 if wtype == "e2m1" else 1  # in an element of the weight
    sf_type, rows, cols = {"bf16": (None, 1, 1), "e4m3": ("float", 128, 128), "e2m1": ("e8m0", 1, 32)}[wtype]

    def sf(t, what, m, c):  # of weight rows m and columns c
        return (_arg(t, what, sf_type, E * (m // rows) * (c // cols)),) if sf_type else ()

    return (_product_ref(product, bind), _arg(x, "x", "bf16", T * H), _arg(topk_idx, "topk_idx", "int32", T * K),
            _arg(topk_weights, "topk_weights", "float", T * K),
            _arg(w1, "w1", wtype, E * M * H // codes), *sf(w1_sf, "w1_sf", M, H),
            _arg(b1, "b1", "float", E * M),
            _arg(w2, "w2", wtype, E * H * I // codes), *sf(w2_sf, "w2_sf", H, I),
            _arg(b2, "b2", "float", E * H),
            _arg(residual, "residual", "bf16", T * H), _arg(out, "out", "bf16", T * H),
            _arg(workspace, "workspace", "bytes", workspace_bytes), workspace_bytes, _stream(stream))


def ep_moe_tokens(problem, product, x, topk_idx, topk_weights, w1, b1, w2, b2, residual, out, workspace,
                  workspace_bytes=None, stream=None, bind=False):
    """The whole expert layer for up to EP_MOE_TOKENS_MAX tokens: up product,
    activation, down product, weighted sum and residual, in two kernels."""
    return _run("ep_moe_tokens", problem, _tokens_ptrs(problem, product, x, topk_idx, topk_weights, w1, None, b1, w2,
        None, b2, residual, out, workspace, workspace_bytes, "bf16", stream, bind), bind)


def ep_moe_tokens_fp8(problem, product, x, topk_idx, topk_weights, w1_fp8, w1_sf, b1, w2_fp8, w2_sf, b2, residual, out,
                      workspace, workspace_bytes=None, stream=None, bind=False):
    """ep_moe_tokens with e4m3 weights and one scale for each 128 x 128 of them."""
    return _run("ep_moe_tokens_fp8", problem, _tokens_ptrs(problem, product, x, topk_idx, topk_weights, w1_fp8, w1_sf,
        b1, w2_fp8, w2_sf, b2, residual, out, workspace, workspace_bytes, "e4m3", stream, bind), bind)


def ep_expert_product_fp4(problem, product, x, expert_count, expert_offset, w_fp4, w_sf, bias=None, residual=None,
                          out=None, stream=None, bind=False):
    """ep_expert_product of up to EP_MOE_TOKENS_MAX tokens with MXFP4 weights:
    e2m1 codes, two a byte, and one e8m0 scale for each 32 of a row."""
    E, C, N, M, rows = _product_sizes(problem, product, expert_count)
    _on_current_device(stream, x, expert_count, expert_offset, w_fp4, w_sf, bias, residual, out)
    return _run("ep_expert_product_fp4", problem, (_product_ref(product, bind), _arg(x, "x", "bf16", rows * C),
        _arg(expert_count, "expert_count", "int32", E), _arg(expert_offset, "expert_offset", "int32", E),
        _arg(w_fp4, "w_fp4", "e2m1", E * M * C // 2), _arg(w_sf, "w_sf", "e8m0", E * M * (C // 32)),
        _arg(bias, "bias", "float", E * M), _arg(residual, "residual", "bf16", rows * N),
        _arg(out, "out", "bf16", rows * N), _stream(stream)), bind)


def ep_moe_tokens_fp4(problem, product, x, topk_idx, topk_weights, w1_fp4, w1_sf, b1, w2_fp4, w2_sf, b2, residual, out,
                      workspace, workspace_bytes=None, stream=None, bind=False):
    """ep_moe_tokens with MXFP4 weights."""
    _on_current_device(stream, x, topk_idx, topk_weights, w1_fp4, w1_sf, b1, w2_fp4, w2_sf, b2, residual, out, workspace)
    return _run("ep_moe_tokens_fp4", problem, _tokens_ptrs(problem, product, x, topk_idx, topk_weights, w1_fp4, w1_sf,
        b1, w2_fp4, w2_sf, b2, residual, out, workspace, workspace_bytes, "e2m1", stream, bind), bind)


def _logits_type(router):
    return "bf16" if router.logits_bf16 else "float"


def _statistics_ptrs(problem, expert_count, token_count, prob_sum, losses, workspace, workspace_bytes):
    E = problem.num_experts
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return (_arg(expert_count, "expert_count", "int32", E), _arg(token_count, "token_count", "int32", 1),
            _arg(prob_sum, "prob_sum", "float", E), _arg(losses, "losses", "float", 2),
            _arg(workspace, "workspace", "bytes", workspace_bytes), workspace_bytes)


def ep_route_workspace_bytes(problem: Problem, router: Router) -> int:
    return load().ep_route_workspace_bytes(ctypes.byref(problem), ctypes.byref(router))


def ep_route(problem, router, logits, bias, token_mask, topk_idx, topk_weights, expert_count=None, token_count=None,
             prob_sum=None, losses=None, workspace=None, workspace_bytes=None, stream=None, bind=False):
    """The router: top-k experts and their weights from the logits, and with
    the last arguments the counts, the balance loss and the z loss."""
    T, _, K, E, _, _, _ = _sizes(problem)
    _on_current_device(stream, logits, bias, token_mask, topk_idx, topk_weights, expert_count, token_count, prob_sum, losses,
                       workspace)
    return _run("ep_route", problem, (_product_ref(router, bind), _arg(logits, "logits", _logits_type(router), T * E),
        _arg(bias, "bias", "float", E), _arg(token_mask, "token_mask", "uint8", T),
        _arg(topk_idx, "topk_idx", "int32", T * K), _arg(topk_weights, "topk_weights", "float", T * K),
        *_statistics_ptrs(problem, expert_count, token_count, prob_sum, losses, workspace, workspace_bytes),
        _stream(stream)), bind)


def ep_balance_loss(problem, router, logits, topk_idx, token_mask, expert_count, token_count, prob_sum, losses,
                    workspace, workspace_bytes=None, stream=None, bind=False):
    """The counts, the balance loss and the z loss of choices made elsewhere."""
    T, _, K, E, _, _, _ = _sizes(problem)
    _on_current_device(stream, logits, topk_idx, token_mask, expert_count, token_count, prob_sum, losses, workspace)
    return _run("ep_balance_loss", problem, (_product_ref(router, bind),
        _arg(logits, "logits", _logits_type(router), T * E), _arg(topk_idx, "topk_idx", "int32", T * K),
        _arg(token_mask, "token_mask", "uint8", T),
        *_statistics_ptrs(problem, expert_count, token_count, prob_sum, losses, workspace, workspace_bytes),
        _stream(stream)), bind)


def ep_route_backward(problem, router, logits, topk_idx, token_mask, expert_count, token_count, dweights, dlosses,
                      dlogits, stream=None, bind=False):
    """The logits' gradient from those of the weights (None: without) and of
    the two losses (None: without)."""
    T, _, K, E, _, _, _ = _sizes(problem)
    _on_current_device(stream, logits, topk_idx, token_mask, expert_count, token_count, dweights, dlosses, dlogits)
    return _run("ep_route_backward", problem, (_product_ref(router, bind),
        _arg(logits, "logits", _logits_type(router), T * E), _arg(topk_idx, "topk_idx", "int32", T * K),
        _arg(token_mask, "token_mask", "uint8", T), _arg(expert_count, "expert_count", "int32", E),
        _arg(token_count, "token_count", "int32", 1), _arg(dweights, "dweights", "float", T * K),
        _arg(dlosses, "dlosses", "float", 2), _arg(dlogits, "dlogits", _logits_type(router), T * E),
        _stream(stream)), bind)


class _BoundGradCall:
    """BoundCall for the calls on gradients: holds their array (and so the tensors)."""

    def __init__(self, name: str, grads: Grads, args: tuple):
        self.name, self.grads = name, grads
        self._fn, self._args = getattr(load(), name), (grads.array, len(grads), *args)

    def __call__(self) -> int:
        return _check(self._fn(*self._args), self.name)


def _run_grads(name: str, grads: Grads, args: tuple, bind: bool):
    call = _BoundGradCall(name, grads, args)
    return call if bind else call()


def ep_grad_workspace_bytes(grads: Grads) -> int:
    return load().ep_grad_workspace_bytes(grads.array, len(grads))


def ep_grad_square_sum(grads, square_sum, workspace, workspace_bytes=None, stream=None, bind=False):
    """square_sum = the sum of all gradients' squares (fp64, on the device);
    ranks with gradients of their own add theirs up before ep_grad_clip."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _on_current_device(stream, square_sum, workspace, *grads.tensors[0][:1])
    return _run_grads("ep_grad_square_sum", grads, (_arg(square_sum, "square_sum", "double", 1),
        _arg(workspace, "workspace", "bytes", workspace_bytes), workspace_bytes, _stream(stream)), bind)


def ep_grad_clip(grads, square_sum, max_norm, norm=None, stream=None, bind=False):
    """out = grad * min(1, max_norm / sqrt(square_sum)), and the norm."""
    _on_current_device(stream, square_sum, norm, *grads.tensors[0][:1])
    return _run_grads("ep_grad_clip", grads, (_arg(square_sum, "square_sum", "double", 1), max_norm,
        _arg(norm, "norm", "float", 1), _stream(stream)), bind)


def ep_read_status(workspace, stream=None) -> int:
    """Synchronises the stream and returns the layout's device status code."""
    return load().ep_read_status(_arg(workspace, "workspace", "bytes", 4), _stream(stream))
