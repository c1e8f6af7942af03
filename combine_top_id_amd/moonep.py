"""Thin ctypes binding of libmoonep.so (the C ABI in include/moonep.h).

Argument marshalling only: torch tensors supply device pointers and the current HIP
stream; every step of the path runs in the library's HIP kernels.  There is no CPU
fallback: if the library is not built, or no GPU is present, calls raise.
"""

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoonep.so")

MOONEP_OK = 0
ROW_ALIGN = 16


class MoonepError(RuntimeError):
    pass


class Sizes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("R", "E", "K", "S", "slots", "E_loc", "C", "G",
                                              "NvS", "P_max")] + \
               [(n, ctypes.c_int64) for n in ("T", "A", "recv_rows", "plan_bytes",
                                              "workspace_bytes")] + \
               [(n, ctypes.c_int32) for n in ("nblk", "blk")] + \
               [(n, ctypes.c_int64) for n in ("o_hdr", "o_load", "o_shed", "o_keep",
                                              "o_home_row", "o_pfirst", "o_pnum", "o_pieces",
                                              "o_slot_expert", "o_off", "o_red", "o_xtab",
                                              "o_ptab", "o_dst_row", "o_w")]


class PlanDesc(ctypes.Structure):
    _fields_ = [("magic", ctypes.c_uint32), ("sz", Sizes), ("dev", ctypes.c_void_p)]


class PlanStats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("status", "bad_index", "n_pieces", "n_replicas",
                                              "n_fallback", "max_pieces_per_rank", "n_red",
                                              "n_shed", "max_load")]


_lib = None


def lib():
    """Load libmoonep.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise MoonepError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    L.moonep_query.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(Sizes)]
    L.moonep_plan.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp, ctypes.POINTER(PlanDesc), vp]
    L.moonep_plan_noalloc.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, ctypes.POINTER(PlanDesc),
                                      vp]
    L.moonep_dispatch.argtypes = [ctypes.POINTER(PlanDesc), vp, i32, vp, vp]
    L.moonep_combine.argtypes = [ctypes.POINTER(PlanDesc), vp, i32, vp, vp]
    L.moonep_reduce_grad.argtypes = [ctypes.POINTER(PlanDesc), vp, vp, i64, vp]
    L.moonep_dispatch_bwd.argtypes = [ctypes.POINTER(PlanDesc), vp, i32, vp, vp]
    L.moonep_combine_bwd.argtypes = [ctypes.POINTER(PlanDesc), vp, vp, i32, vp, vp, vp]
    L.moonep_dispatch_staged.argtypes = [ctypes.POINTER(PlanDesc), vp, i32, vp, vp, vp]
    L.moonep_combine_staged.argtypes = [ctypes.POINTER(PlanDesc), vp, i32, vp, vp, vp]
    L.moonep_prefetch_weight.argtypes = [ctypes.POINTER(PlanDesc), vp, i64, vp, vp]
    L.moonep_expert_stub.argtypes = [ctypes.POINTER(PlanDesc), vp, vp, vp, vp, i64, i32, vp, vp]
    PD, f32 = ctypes.POINTER(PlanDesc), ctypes.c_float
    L.moonep_expert_ffn.argtypes = [PD, vp, i32, i32, i32, vp, vp, i64, vp, vp, vp, vp]
    L.moonep_expert_ffn_bwd_data.argtypes = [PD, vp, vp, i32, i32, i32, vp, vp, i64, vp, vp, vp]
    L.moonep_expert_ffn_bwd_weight.argtypes = [PD, vp, vp, vp, vp, i32, i32, vp, vp, i64, i32, vp]
    L.moonep_expert_tile.argtypes = [PD, i32, i32, i32, ctypes.POINTER(ctypes.c_int32)]
    L.moonep_rmsnorm.argtypes = [vp, vp, vp, f32, i64, i32, vp, vp, vp, vp]
    L.moonep_rmsnorm_q8.argtypes = [vp, vp, vp, f32, i64, i32, vp, vp, vp, vp]
    L.moonep_q8_unpack.argtypes = [vp, i64, i32, vp, vp]
    L.moonep_rmsnorm_bwd.argtypes = [vp, vp, vp, vp, vp, i64, i32, vp, vp, vp, vp]
    L.moonep_q8_row_bytes.argtypes = [i32]
    L.moonep_router.argtypes = [vp, i32, vp, i64, i32, i32, i32, i32, i32, i32, f32, vp, vp, vp]
    L.moonep_router_bwd.argtypes = [vp, i32, vp, vp, i64, i32, i32, i32, i32, f32, vp, vp]
    L.moonep_w4_slab_bytes.argtypes = [i32, i32]
    L.moonep_w4_pack.argtypes = [vp, i64, i64, i32, i32, vp, i64, vp]
    L.moonep_w4_unpack.argtypes = [vp, i64, i64, i32, i32, vp, i64, vp]
    L.moonep_expert_tile_w4.argtypes = [PD, i32, i32, i32, i32, ctypes.POINTER(ctypes.c_int32)]
    L.moonep_expert_ffn_w4.argtypes = [PD, vp, i32, i32, i32, vp, vp, i64, vp, vp, vp, vp]
    L.moonep_expert_ffn_w4q8.argtypes = [PD, vp, i32, i32, i32, vp, vp, i64, vp, vp, vp]
    L.moonep_rmsnorm_bwd_workspace.argtypes = [i64, i32]
    for f in ("moonep_q8_row_bytes", "moonep_rmsnorm_bwd_workspace", "moonep_w4_slab_bytes"):
        getattr(L, f).restype = i64
    L.moonep_plan_status.argtypes = [ctypes.POINTER(PlanDesc), ctypes.POINTER(PlanStats), vp]
    L.moonep_strerror.argtypes = [i32]
    L.moonep_strerror.restype = ctypes.c_char_p
    for f in ("moonep_query", "moonep_plan", "moonep_plan_noalloc", "moonep_dispatch",
              "moonep_combine",
              "moonep_reduce_grad", "moonep_plan_status", "moonep_dispatch_bwd",
              "moonep_combine_bwd", "moonep_prefetch_weight", "moonep_expert_stub",
              "moonep_dispatch_staged", "moonep_combine_staged", "moonep_expert_ffn",
              "moonep_expert_ffn_bwd_data", "moonep_expert_ffn_bwd_weight", "moonep_expert_tile",
              "moonep_rmsnorm", "moonep_rmsnorm_q8", "moonep_q8_unpack", "moonep_rmsnorm_bwd",
              "moonep_w4_pack", "moonep_w4_unpack", "moonep_expert_ffn_w4", "moonep_expert_ffn_w4q8",
              "moonep_expert_tile_w4", "moonep_router", "moonep_router_bwd"):
        getattr(L, f).restype = i32
    _lib = L
    return L


EXPORTS = ("moonep_query", "moonep_plan", "moonep_plan_noalloc", "moonep_dispatch",
           "moonep_combine",
           "moonep_reduce_grad", "moonep_plan_status", "moonep_strerror",
           "moonep_dispatch_bwd", "moonep_combine_bwd", "moonep_prefetch_weight",
           "moonep_expert_stub", "moonep_dispatch_staged", "moonep_combine_staged",
           "moonep_expert_ffn", "moonep_expert_ffn_bwd_data", "moonep_expert_ffn_bwd_weight",
           "moonep_expert_tile", "moonep_rmsnorm", "moonep_rmsnorm_q8", "moonep_q8_row_bytes", "moonep_q8_unpack",
           "moonep_rmsnorm_bwd_workspace", "moonep_rmsnorm_bwd", "moonep_w4_slab_bytes", "moonep_w4_pack",
           "moonep_w4_unpack", "moonep_expert_ffn_w4", "moonep_expert_ffn_w4q8", "moonep_expert_tile_w4",
           "moonep_router", "moonep_router_bwd")

ACTIVATIONS = {"silu": 0, "gelu": 1}
SCORES = {"softmax": 0, "sigmoid": 1}
LOGITS = {torch.float32: 0, torch.bfloat16: 1}
PRODUCTS = ("gate_up", "down", "g_gate_up", "g_rows", "g_weights")


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _check(rc):
    if rc != MOONEP_OK:
        raise MoonepError(f"moonep error {rc}: {lib().moonep_strerror(rc).decode()}")


def _stream(stream, device):
    """The HIP stream handle to enqueue on: `stream`, else the current stream of the
    tensors' device (not of whichever device happens to be current)."""
    if stream is None:
        # the handle itself: building a Stream object around it takes longer than some kernels
        return _raw_stream(device.index)
    if stream.device != device:
        raise MoonepError(f"stream is on {stream.device}, the tensors on {device}")
    return stream.cuda_stream


def _dev(t, dtype, name, device=None):
    """The device address of `t`, checked."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise MoonepError(f"{name} must be a GPU tensor")
    if device is not None and t.get_device() != device.index:
        raise MoonepError(f"{name} is on {t.device}, the plan on {device}")
    if t.dtype is not dtype:
        raise MoonepError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise MoonepError(f"{name} must be contiguous")
    return t.data_ptr()


def _run(f, device, *args):
    """One call of the library, with `device` the current one while it launches."""
    if torch.cuda.current_device() == device.index:
        _check(f(*args))
    else:
        with torch.cuda.device(device):
            _check(f(*args))


def moonep_query(R, E, K, S, slots) -> Sizes:
    s = Sizes()
    _check(lib().moonep_query(R, E, K, S, slots, ctypes.byref(s)))
    return s


class Plan:
    """A plan: host descriptor + the device blob it describes (+ its workspace)."""

    def __init__(self, sizes, blob, workspace):
        self.sz = sizes
        self.blob = blob
        self.workspace = workspace
        self.desc = PlanDesc()

    @property
    def NvS(self):
        return self.sz.NvS

    def array(self, name, count):
        """A view of one int32 array of the device blob (offset field `o_<name>`)."""
        o = getattr(self.sz, "o_" + name)
        return self.blob[o:o + count]

    @property
    def dst_row(self):
        return self.array("dst_row", self.sz.A).view(self.sz.T, self.sz.K)

    @property
    def weights(self):
        return self.array("w", self.sz.A).view(torch.float32).view(self.sz.T, self.sz.K)


def _blob(nbytes, device, zero=False):
    # int32 elements; torch's caching allocator returns 256-byte aligned blocks
    n = (nbytes + 3) // 4
    t = (torch.zeros if zero else torch.empty)(n, dtype=torch.int32, device=device)
    assert t.data_ptr() % 256 == 0
    return t


def moonep_plan(topk_ids, topk_w, R, E, K, S, slots, plan=None, stream=None) -> Plan:
    """Enqueue the planning kernels; returns the Plan (reusable by dispatch, combine and
    reduce).  Pass `plan` to reuse its blob and workspace (same sizes)."""
    sz = moonep_query(R, E, K, S, slots)
    ids_p = _dev(topk_ids, torch.int32, "topk_ids")
    w_p = _dev(topk_w, torch.float32, "topk_w", topk_ids.device)
    if topk_ids.numel() != sz.A or topk_w.numel() != sz.A:
        raise MoonepError("topk_ids / topk_w must hold R*S*K elements")
    if plan is None or plan.workspace is None or plan.sz.plan_bytes != sz.plan_bytes or \
            plan.sz.workspace_bytes != sz.workspace_bytes:
        # the workspace starts zero-filled; every plan call leaves it so
        plan = Plan(sz, _blob(sz.plan_bytes, topk_ids.device),
                    _blob(sz.workspace_bytes, topk_ids.device, zero=True))
    plan.sz = sz
    _check(lib().moonep_plan(ids_p, w_p, R, E, K, S, slots,
                             ctypes.c_void_p(plan.blob.data_ptr()),
                             ctypes.c_void_p(plan.workspace.data_ptr()),
                             ctypes.byref(plan.desc), _stream(stream, topk_ids.device)))
    return plan


def moonep_plan_noalloc(topk_ids, topk_w, R, E, K, S, slots, plan=None, stream=None) -> Plan:
    """moonep_plan through the entry point that allocates nothing: the planning workspace is
    the library's static per-GPU array (at most MOONEP_NOALLOC_WORKSPACE_MAX bytes).  The
    plan blob is the caller's (`plan`'s, else one allocated here, outside the C call)."""
    sz = moonep_query(R, E, K, S, slots)
    D = topk_ids.device
    ids_p = _dev(topk_ids, torch.int32, "topk_ids")
    w_p = _dev(topk_w, torch.float32, "topk_w", D)
    if topk_ids.numel() != sz.A or topk_w.numel() != sz.A:
        raise MoonepError("topk_ids / topk_w must hold R*S*K elements")
    if plan is None or plan.sz.plan_bytes != sz.plan_bytes or plan.blob.device != D:
        plan = Plan(sz, _blob(sz.plan_bytes, D), None)
    plan.sz = sz
    with torch.cuda.device(D):       # the library uses the current device's array
        _check(lib().moonep_plan_noalloc(ids_p, w_p, R, E, K, S, slots,
                                         ctypes.c_void_p(plan.blob.data_ptr()),
                                         ctypes.byref(plan.desc), _stream(stream, D)))
    return plan


def moonep_dispatch(plan: Plan, x, recv=None, stream=None):
    """recv[dst_row[t, k]] = x[t]; x is bf16 [T, H]; returns recv bf16 [R*NvS, H]."""
    D = plan.blob.device
    H = x.shape[-1]
    if x.numel() != plan.sz.T * H:
        raise MoonepError("x must be [T, H]")
    if recv is None:
        recv = torch.empty(plan.sz.recv_rows, H, dtype=torch.bfloat16, device=x.device)
    if recv.numel() != plan.sz.recv_rows * H:
        raise MoonepError("recv must be [R*NvS, H]")
    _check(lib().moonep_dispatch(ctypes.byref(plan.desc), _dev(x, torch.bfloat16, "x", D), H,
                                 _dev(recv, torch.bfloat16, "recv", D), _stream(stream, D)))
    return recv


def moonep_combine(plan: Plan, y, out=None, stream=None):
    """out[t] = bf16(sum_k w[t,k] * y[dst_row[t,k]]); y bf16 [R*NvS, H] -> out bf16 [T, H]."""
    D = plan.blob.device
    H = y.shape[-1]
    if y.numel() != plan.sz.recv_rows * H:
        raise MoonepError("y must be [R*NvS, H]")
    if out is None:
        out = torch.empty(plan.sz.T, H, dtype=torch.bfloat16, device=y.device)
    if out.numel() != plan.sz.T * H:
        raise MoonepError("out must be [T, H]")
    _check(lib().moonep_combine(ctypes.byref(plan.desc), _dev(y, torch.bfloat16, "y", D), H,
                                _dev(out, torch.bfloat16, "out", D), _stream(stream, D)))
    return out


def _stage(plan, H, stage, device):
    if stage is None:
        stage = torch.empty(plan.sz.A, H, dtype=torch.bfloat16, device=device)
    if stage.numel() != plan.sz.A * H:
        raise MoonepError("stage must be [T*K, H]")
    return stage


def moonep_dispatch_staged(plan: Plan, x, recv=None, stage=None, stream=None):
    """Non-zero-copy dispatch: x -> stage (arrival order) -> recv (epilogue copy)."""
    D = plan.blob.device
    H = x.shape[-1]
    if x.numel() != plan.sz.T * H:
        raise MoonepError("x must be [T, H]")
    stage = _stage(plan, H, stage, x.device)
    if recv is None:
        recv = torch.empty(plan.sz.recv_rows, H, dtype=torch.bfloat16, device=x.device)
    if recv.numel() != plan.sz.recv_rows * H:
        raise MoonepError("recv must be [R*NvS, H]")
    _check(lib().moonep_dispatch_staged(ctypes.byref(plan.desc), _dev(x, torch.bfloat16, "x", D), H,
                                        _dev(stage, torch.bfloat16, "stage", D),
                                        _dev(recv, torch.bfloat16, "recv", D), _stream(stream, D)))
    return recv


def moonep_combine_staged(plan: Plan, y, out=None, stage=None, stream=None):
    """Non-zero-copy combine: y -> stage (prologue copy) -> weighted sum -> out."""
    D = plan.blob.device
    H = y.shape[-1]
    if y.numel() != plan.sz.recv_rows * H:
        raise MoonepError("y must be [R*NvS, H]")
    stage = _stage(plan, H, stage, y.device)
    if out is None:
        out = torch.empty(plan.sz.T, H, dtype=torch.bfloat16, device=y.device)
    if out.numel() != plan.sz.T * H:
        raise MoonepError("out must be [T, H]")
    _check(lib().moonep_combine_staged(ctypes.byref(plan.desc), _dev(y, torch.bfloat16, "y", D), H,
                                       _dev(stage, torch.bfloat16, "stage", D),
                                       _dev(out, torch.bfloat16, "out", D), _stream(stream, D)))
    return out


def moonep_dispatch_bwd(plan: Plan, g_recv, gx=None, stream=None):
    """gx[t] = bf16(sum_k g_recv[dst_row[t,k]]); g_recv bf16 [R*NvS, H] -> gx bf16 [T, H]."""
    D = plan.blob.device
    H = g_recv.shape[-1]
    if g_recv.numel() != plan.sz.recv_rows * H:
        raise MoonepError("g_recv must be [R*NvS, H]")
    if gx is None:
        gx = torch.empty(plan.sz.T, H, dtype=torch.bfloat16, device=g_recv.device)
    if gx.numel() != plan.sz.T * H:
        raise MoonepError("gx must be [T, H]")
    _check(lib().moonep_dispatch_bwd(ctypes.byref(plan.desc),
                                     _dev(g_recv, torch.bfloat16, "g_recv", D),
                                     H, _dev(gx, torch.bfloat16, "gx", D), _stream(stream, D)))
    return gx


def moonep_combine_bwd(plan: Plan, dout, y, g_y=None, dw=None, stream=None):
    """g_y[dst_row[t,k]] = bf16(w[t,k] * dout[t]); dw[t,k] = <dout[t], y[dst_row[t,k]]>.
    dout bf16 [T, H], y bf16 [R*NvS, H]; returns (g_y bf16 [R*NvS, H], dw fp32 [T, K])."""
    D = plan.blob.device
    H = dout.shape[-1]
    if dout.numel() != plan.sz.T * H or y.numel() != plan.sz.recv_rows * H:
        raise MoonepError("dout must be [T, H] and y [R*NvS, H]")
    if g_y is None:
        g_y = torch.empty(plan.sz.recv_rows, H, dtype=torch.bfloat16, device=dout.device)
    if dw is None:
        dw = torch.empty(plan.sz.T, plan.sz.K, dtype=torch.float32, device=dout.device)
    if g_y.numel() != plan.sz.recv_rows * H or dw.numel() != plan.sz.T * plan.sz.K:
        raise MoonepError("g_y must be [R*NvS, H] and dw [T, K]")
    _check(lib().moonep_combine_bwd(ctypes.byref(plan.desc), _dev(dout, torch.bfloat16, "dout", D),
                                    _dev(y, torch.bfloat16, "y", D), H,
                                    _dev(g_y, torch.bfloat16, "g_y", D),
                                    _dev(dw, torch.float32, "dw", D), _stream(stream, D)))
    return g_y, dw


def moonep_prefetch_weight(plan: Plan, home_w, slot_w=None, stream=None):
    """slot_w[r, slot] = home_w[e] for every slot piece; home_w bf16 [E, W_el] ->
    slot_w bf16 [R, slots, W_el]."""
    D = plan.blob.device
    W_el = home_w.shape[-1]
    if home_w.numel() != plan.sz.E * W_el:
        raise MoonepError("home_w must be [E, W_el]")
    if slot_w is None:
        slot_w = torch.empty(plan.sz.R, plan.sz.slots, W_el, dtype=torch.bfloat16,
                             device=home_w.device)
    if slot_w.numel() != plan.sz.R * plan.sz.slots * W_el:
        raise MoonepError("slot_w must be [R, slots, W_el]")
    sp = _dev(slot_w, torch.bfloat16, "slot_w", D) if slot_w.numel() else ctypes.c_void_p(0)
    _check(lib().moonep_prefetch_weight(ctypes.byref(plan.desc),
                                        _dev(home_w, torch.bfloat16, "home_w", D), W_el, sp,
                                        _stream(stream, D)))
    return slot_w


def moonep_expert_stub(plan: Plan, topk_ids, recv, home_w, slot_w, y=None, stream=None):
    """y[row] = bf16(recv[row] * W[:H]) with W the weight slab the row's group reads."""
    D = plan.blob.device
    H = recv.shape[-1]
    W_el = home_w.shape[-1]
    if topk_ids.numel() != plan.sz.A:
        raise MoonepError("topk_ids must hold R*S*K elements")
    if recv.numel() != plan.sz.recv_rows * H:
        raise MoonepError("recv must be [R*NvS, H]")
    if home_w.numel() != plan.sz.E * W_el or slot_w.numel() != plan.sz.R * plan.sz.slots * W_el:
        raise MoonepError("home_w must be [E, W_el] and slot_w [R, slots, W_el]")
    if y is None:
        y = torch.empty_like(recv)
    if y.numel() != recv.numel():
        raise MoonepError("y must be [R*NvS, H]")
    sp = _dev(slot_w, torch.bfloat16, "slot_w", D) if slot_w.numel() else ctypes.c_void_p(0)
    _check(lib().moonep_expert_stub(ctypes.byref(plan.desc),
                                    _dev(topk_ids, torch.int32, "topk_ids", D),
                                    _dev(recv, torch.bfloat16, "recv", D),
                                    _dev(home_w, torch.bfloat16, "home_w", D), sp, W_el, H,
                                    _dev(y, torch.bfloat16, "y", D), _stream(stream, D)))
    return y


def moonep_reduce_grad(plan: Plan, home_grad, rep_grad, stream=None):
    """home_grad[e] += replica slabs of e (in place); home fp32 [E, G_el], rep fp32
    [R, slots, G_el]."""
    D = plan.blob.device
    G_el = home_grad.shape[-1]
    if home_grad.numel() != plan.sz.E * G_el:
        raise MoonepError("home_grad must be [E, G_el]")
    if rep_grad.numel() != plan.sz.R * plan.sz.slots * G_el:
        raise MoonepError("rep_grad must be [R, slots, G_el]")
    rep_p = _dev(rep_grad, torch.float32, "rep_grad", D) if rep_grad.numel() else ctypes.c_void_p(0)
    _check(lib().moonep_reduce_grad(ctypes.byref(plan.desc),
                                    _dev(home_grad, torch.float32, "home_grad", D), rep_p, G_el,
                                    _stream(stream, D)))
    return home_grad


def _bytes(n):
    """The result of a host-only size call: bytes, or a negative error code."""
    if n < 0:
        _check(int(n))
    return n


def _on_its_stream(f):
    """f, allocating what it is not given on the stream that it is told to use: memory of
    another stream could be handed on there (a workspace at once) while the call still runs.
    The stream is given by its name."""
    @functools.wraps(f)
    def call(*args, stream=None, **kwargs):
        if stream is None:
            return f(*args, **kwargs)
        with torch.cuda.stream(stream):
            return f(*args, stream=stream, **kwargs)
    return call


def _rows(t, dtype, name, rows, cols, device, like):
    """`t` checked to be [rows, cols] (its device pointer comes second), allocated next to
    `like` if it is None."""
    if t is None:
        t = like.new_empty((rows, cols)) if like.dtype is dtype else \
            torch.empty(rows, cols, dtype=dtype, device=like.device)
    p = _dev(t, dtype, name, device)
    if t.numel() != rows * cols:
        raise MoonepError(f"{name} must be [{rows}, {cols}]")
    return t, p


def _slabs(plan, home, slot, el, dtype, names):
    """Device pointers and the pitch of an [E, pitch] and an [R, slots, pitch] array of
    experts' slabs of at least `el` elements."""
    D = plan.blob.device
    hp = _dev(home, dtype, names[0], D)
    pitch = home.shape[-1]
    if home.numel() != plan.sz.E * pitch or pitch < el:
        raise MoonepError(f"{names[0]} must be [E, {el} or more]")
    n = plan.sz.R * plan.sz.slots * pitch
    if (slot.numel() if slot is not None else 0) != n:
        raise MoonepError(f"{names[1]} must be [R, slots, {pitch}]")
    return hp, (_dev(slot, dtype, names[1], D) if n else None), pitch


def _act(act):
    if act not in ACTIVATIONS:
        raise MoonepError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


@_on_its_stream
def moonep_expert_ffn(plan: Plan, recv, home_w, slot_w, I, act="silu", save=False, h=None, gu=None,
                      y=None, *, stream=None):
    """The gated feed-forward experts: y[row] = Wd (act(Wg x) * (Wu x)) with x = recv[row] and
    the weights of the row's group.  recv bf16 [R*NvS, H]; home_w bf16 [E, W_el], an
    expert's slab being gate [I, H], up [I, H], down [H, I]; slot_w bf16 [R, slots, W_el].
    Returns (y, h, gu): y bf16 [R*NvS, H], h bf16 [R*NvS, I], and, where `save` is true or
    a buffer is passed, the gate and up rows gu bf16 [R*NvS, 2*I] (else None).  The
    gradients need h and gu."""
    D, n = plan.blob.device, plan.sz.recv_rows
    H = recv.shape[-1]
    _, rp = _rows(recv, torch.bfloat16, "recv", n, H, D, recv)
    wp, sp, W_el = _slabs(plan, home_w, slot_w, 3 * I * H, torch.bfloat16, ("home_w", "slot_w"))
    h, hp = _rows(h, torch.bfloat16, "h", n, I, D, recv)
    y, yp = _rows(y, torch.bfloat16, "y", n, H, D, recv)
    gp = None
    if save or gu is not None:
        gu, gp = _rows(gu, torch.bfloat16, "gu", n, 2 * I, D, recv)
    _run(lib().moonep_expert_ffn, D, ctypes.byref(plan.desc), rp, H, I, _act(act), wp, sp, W_el, gp, hp,
         yp, _stream(stream, D))
    return y, h, gu


@_on_its_stream
def moonep_expert_ffn_bwd_data(plan: Plan, g_y, gu, home_w, slot_w, I, act="silu", g_gu=None,
                               g_recv=None, *, stream=None):
    """Gradient of moonep_expert_ffn with respect to the rows, from g_y bf16 [R*NvS, H] and the
    saved gu.  Returns (g_recv bf16 [R*NvS, H], g_gu bf16 [R*NvS, 2*I]); g_gu may be gu."""
    D, n = plan.blob.device, plan.sz.recv_rows
    H = g_y.shape[-1]
    _, yp = _rows(g_y, torch.bfloat16, "g_y", n, H, D, g_y)
    _, gp = _rows(gu, torch.bfloat16, "gu", n, 2 * I, D, g_y) if gu is not None else (None, None)
    if gp is None:
        raise MoonepError("gu must be a GPU tensor")
    wp, sp, W_el = _slabs(plan, home_w, slot_w, 3 * I * H, torch.bfloat16, ("home_w", "slot_w"))
    g_gu, ggp = _rows(g_gu, torch.bfloat16, "g_gu", n, 2 * I, D, g_y)
    g_recv, grp = _rows(g_recv, torch.bfloat16, "g_recv", n, H, D, g_y)
    _run(lib().moonep_expert_ffn_bwd_data, D, ctypes.byref(plan.desc), yp, gp, H, I, _act(act), wp, sp,
         W_el, ggp, grp, _stream(stream, D))
    return g_recv, g_gu


@_on_its_stream
def moonep_expert_ffn_bwd_weight(plan: Plan, recv, g_y, h, g_gu, home_grad=None, rep_grad=None,
                                 accumulate=False, *, stream=None):
    """Gradient of moonep_expert_ffn with respect to the weights: home_grad fp32 [E, G_el]
    (overwritten, or added to with `accumulate`) and rep_grad fp32 [R, slots, G_el]
    (overwritten in the slots the plan uses), laid out as the weights' slabs;
    moonep_reduce_grad then adds the replicas to their homes.  Returns both."""
    D, n = plan.blob.device, plan.sz.recv_rows
    if h is None or g_y is None or g_gu is None:
        raise MoonepError("g_y, h and g_gu must be GPU tensors")
    H, I = recv.shape[-1], h.shape[-1]
    _, rp = _rows(recv, torch.bfloat16, "recv", n, H, D, recv)
    _, yp = _rows(g_y, torch.bfloat16, "g_y", n, H, D, recv)
    _, hp = _rows(h, torch.bfloat16, "h", n, I, D, recv)
    _, gp = _rows(g_gu, torch.bfloat16, "g_gu", n, 2 * I, D, recv)
    if home_grad is None:
        if accumulate:
            raise MoonepError("accumulate needs a home_grad to add to")
        home_grad = torch.empty(plan.sz.E, 3 * I * H, dtype=torch.float32, device=recv.device)
    if rep_grad is None:
        rep_grad = torch.empty(plan.sz.R, plan.sz.slots, home_grad.shape[-1], dtype=torch.float32,
                               device=recv.device)
    wp, sp, G_el = _slabs(plan, home_grad, rep_grad, 3 * I * H, torch.float32, ("home_grad", "rep_grad"))
    _run(lib().moonep_expert_ffn_bwd_weight, D, ctypes.byref(plan.desc), rp, yp, hp, gp, H, I, wp, sp, G_el,
         int(bool(accumulate)), _stream(stream, D))
    return home_grad, rep_grad


def moonep_expert_tile(plan: Plan, H, I, product):
    """The tile that a product of the experts' calls ("gate_up" or "down" of the forward pass,
    "g_gate_up" or "g_rows" of the rows' gradient, "g_weights") is computed in: results along
    an output row, output rows, and whether the results are written past the caches."""
    if product not in PRODUCTS:
        raise MoonepError(f"product must be one of {PRODUCTS}, got {product!r}")
    tile = (ctypes.c_int32 * 3)()
    _check(lib().moonep_expert_tile(ctypes.byref(plan.desc), H, I, PRODUCTS.index(product), tile))
    return tile[0], tile[1], bool(tile[2])


def _norm_args(x, gamma, res, h, rstd, stats):
    """The checked arguments that the norm's two forms share."""
    xp = _dev(x, torch.bfloat16, "x")
    D, H = x.device, x.shape[-1]
    T = x.numel() // H if H else 0
    none = None
    gp = _dev(gamma, torch.bfloat16, "gamma", D)
    if gamma.numel() != H:
        raise MoonepError("gamma must be [H]")
    rp = _rows(res, torch.bfloat16, "res", T, H, D, x)[1] if res is not None else none
    if h is not None or res is not None:
        h, hp = _rows(h, torch.bfloat16, "h", T, H, D, x)
    else:
        h, hp = x, none                  # without a residual the stream is x itself
    sp = none
    if stats or rstd is not None:
        if rstd is None:
            rstd = torch.empty(T, dtype=torch.float32, device=D)
        sp = _dev(rstd, torch.float32, "rstd", D)
        if rstd.numel() != T:
            raise MoonepError("rstd must be [T]")
    return D, T, H, xp, rp, gp, h, hp, rstd, sp


@_on_its_stream
def moonep_rmsnorm(x, gamma, eps=1e-6, res=None, out=None, h=None, rstd=None, stats=True, *, stream=None):
    """h = bf16(x + res), out = bf16(h * rstd * gamma), rstd = 1 / sqrt(mean(h^2) + eps), row by
    row.  x, res bf16 [T, H], gamma bf16 [H].  Returns (out, h, rstd): h is x where there is
    no residual and no buffer for it, rstd (fp32 [T]) is None where `stats` is false."""
    D, T, H, xp, rp, gp, h, hp, rstd, sp = _norm_args(x, gamma, res, h, rstd, stats)
    if out is None:
        out = torch.empty_like(x)
    op = _rows(out, torch.bfloat16, "out", T, H, D, x)[1]
    _run(lib().moonep_rmsnorm, D, xp, rp, gp, eps, T, H, op, hp, sp, _stream(stream, D))
    return out, h, rstd


def moonep_q8_row_bytes(H):
    """Bytes of a row of H elements in 8 bits: codes, a scale for 32 of them, padding to 16."""
    return _bytes(lib().moonep_q8_row_bytes(H))


@_on_its_stream
def moonep_rmsnorm_q8(x, gamma, eps=1e-6, res=None, rows=None, h=None, rstd=None, stats=True, *, stream=None):
    """moonep_rmsnorm with its output as 8-bit rows, uint8 [T, moonep_q8_row_bytes(H)].
    `rows.view(torch.bfloat16)` is what moonep_dispatch moves.  Returns (rows, h, rstd)."""
    D, T, H, xp, rp, gp, h, hp, rstd, sp = _norm_args(x, gamma, res, h, rstd, stats)
    rows, op = _rows(rows, torch.uint8, "rows", T, moonep_q8_row_bytes(H), D, x)
    _run(lib().moonep_rmsnorm_q8, D, xp, rp, gp, eps, T, H, op, hp, sp, _stream(stream, D))
    return rows, h, rstd


@_on_its_stream
def moonep_q8_unpack(rows, H, out=None, *, stream=None):
    """8-bit rows (uint8 [N, moonep_q8_row_bytes(H)], or the same bytes as bf16 elements, as the
    dispatch returns them) expanded to bf16 [N, H]."""
    rb = moonep_q8_row_bytes(H)
    if isinstance(rows, torch.Tensor) and rows.dtype == torch.bfloat16 and rows.is_contiguous():
        rows = rows.view(torch.uint8)
    rp = _dev(rows, torch.uint8, "rows")
    if rows.numel() % rb:
        raise MoonepError(f"rows must be [N, {rb}] bytes")
    N, D = rows.numel() // rb, rows.device
    out, op = _rows(out, torch.bfloat16, "out", N, H, D, rows)
    _run(lib().moonep_q8_unpack, D, rp, N, H, op, _stream(stream, D))
    return out


@_on_its_stream
def moonep_rmsnorm_bwd(g_out, h, gamma, rstd, g_h=None, g_x=None, g_gamma=None, workspace=None, *,
                       stream=None):
    """Backward of the norm from the stored h bf16 [T, H] and rstd fp32 [T]; g_h, if given, is
    the gradient that reaches h past the norm.  Returns (g_x bf16 [T, H], the gradient of x
    and of res; g_gamma fp32 [H])."""
    op = _dev(g_out, torch.bfloat16, "g_out")
    D, H = g_out.device, g_out.shape[-1]
    T = g_out.numel() // H if H else 0
    _, hp = _rows(h, torch.bfloat16, "h", T, H, D, g_out)
    gp = _dev(gamma, torch.bfloat16, "gamma", D)
    sp = _dev(rstd, torch.float32, "rstd", D)
    if gamma.numel() != H or rstd.numel() != T:
        raise MoonepError("gamma must be [H] and rstd [T]")
    ghp = _rows(g_h, torch.bfloat16, "g_h", T, H, D, g_out)[1] if g_h is not None else None
    g_x, xp = _rows(g_x, torch.bfloat16, "g_x", T, H, D, g_out)
    g_gamma, ggp = _rows(g_gamma, torch.float32, "g_gamma", 1, H, D, g_out)
    need = _bytes(lib().moonep_rmsnorm_bwd_workspace(T, H))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=D)
    wp = _dev(workspace, torch.uint8, "workspace", D)
    if workspace.numel() < need:
        raise MoonepError(f"workspace must hold {need} bytes")
    _run(lib().moonep_rmsnorm_bwd, D, op, hp, gp, sp, ghp, T, H, wp, xp, ggp, _stream(stream, D))
    return g_x, g_gamma.view(H)


def moonep_w4_slab_bytes(H, I):
    """Bytes of an expert's slab in 4 bits."""
    return _bytes(lib().moonep_w4_slab_bytes(H, I))


def _row_pitch(t, dtype, name, device=None):
    """Device pointer, rows and columns of a two-dimensional `t`."""
    p = _dev(t, dtype, name, device)
    if t.dim() != 2:
        raise MoonepError(f"{name} must have two dimensions")
    return p, t.shape[0], t.shape[1]


@_on_its_stream
def moonep_w4_pack(w, H, I, out=None, *, stream=None):
    """bf16 slabs [n, W_el] (gate [I, H], up [I, H], down [H, I], as moonep_expert_ffn takes them) in
    4 bits with a power of two for 32: uint8 [n, moonep_w4_slab_bytes(H, I)], or `out`, whose
    rows may be longer.  `out.view(torch.bfloat16)` is what moonep_prefetch_weight moves."""
    wp, n, W_el = _row_pitch(w, torch.bfloat16, "w")
    D, need = w.device, moonep_w4_slab_bytes(H, I)
    if out is None:
        out = torch.empty(n, need, dtype=torch.uint8, device=D)
    op, m, pitch = _row_pitch(out, torch.uint8, "out", D)
    if m != n:
        raise MoonepError(f"out must be [{n}, {need} or more]")
    _run(lib().moonep_w4_pack, D, wp, W_el, n, H, I, op, pitch, _stream(stream, D))
    return out


@_on_its_stream
def moonep_w4_unpack(w4, H, I, out=None, *, stream=None):
    """Slabs in 4 bits (uint8 [n, W_bytes]) expanded exactly to bf16 [n, 3*I*H], or `out`, whose
    rows may be longer: what moonep_expert_ffn and moonep_expert_ffn_bwd_data take."""
    wp, n, pitch = _row_pitch(w4, torch.uint8, "w4")
    D = w4.device
    if out is None:
        out = torch.empty(n, 3 * I * H, dtype=torch.bfloat16, device=D)
    op, m, W_el = _row_pitch(out, torch.bfloat16, "out", D)
    if m != n:
        raise MoonepError(f"out must be [{n}, {3 * I * H} or more]")
    _run(lib().moonep_w4_unpack, D, wp, pitch, n, H, I, op, W_el, _stream(stream, D))
    return out


@_on_its_stream
def moonep_expert_ffn_w4(plan: Plan, recv, home_w4, slot_w4, I, act="silu", save=False, h=None, gu=None,
                         y=None, *, stream=None):
    """moonep_expert_ffn with weights in 4 bits: home_w4 uint8 [E, W_bytes] (moonep_w4_pack's), slot_w4
    uint8 [R, slots, W_bytes].  Rows, results and what is saved are as there."""
    D, n = plan.blob.device, plan.sz.recv_rows
    H = recv.shape[-1]
    _, rp = _rows(recv, torch.bfloat16, "recv", n, H, D, recv)
    wp, sp, pitch = _slabs(plan, home_w4, slot_w4, moonep_w4_slab_bytes(H, I), torch.uint8, ("home_w4", "slot_w4"))
    h, hp = _rows(h, torch.bfloat16, "h", n, I, D, recv)
    y, yp = _rows(y, torch.bfloat16, "y", n, H, D, recv)
    gp = None
    if save or gu is not None:
        gu, gp = _rows(gu, torch.bfloat16, "gu", n, 2 * I, D, recv)
    _run(lib().moonep_expert_ffn_w4, D, ctypes.byref(plan.desc), rp, H, I, _act(act), wp, sp, pitch, gp, hp, yp,
         _stream(stream, D))
    return y, h, gu


@_on_its_stream
def moonep_expert_ffn_w4q8(plan: Plan, rows, home_w4, slot_w4, H, I, act="silu", h=None, y=None, *, stream=None):
    """moonep_expert_ffn with weights in 4 bits and rows in 8: rows uint8 [R*NvS, moonep_q8_row_bytes(H)]
    (moonep_rmsnorm_q8's, dispatched; the same bytes as bf16 elements are taken too).  Returns (y bf16
    [R*NvS, H], h uint8 [R*NvS, moonep_q8_row_bytes(I)])."""
    D, n = plan.blob.device, plan.sz.recv_rows
    if isinstance(rows, torch.Tensor) and rows.dtype == torch.bfloat16 and rows.is_contiguous():
        rows = rows.view(torch.uint8)
    _, rp = _rows(rows, torch.uint8, "rows", n, moonep_q8_row_bytes(H), D, rows)
    wp, sp, pitch = _slabs(plan, home_w4, slot_w4, moonep_w4_slab_bytes(H, I), torch.uint8, ("home_w4", "slot_w4"))
    h, hp = _rows(h, torch.uint8, "h", n, moonep_q8_row_bytes(I), D, rows)
    y, yp = _rows(y, torch.bfloat16, "y", n, H, D, rows)
    _run(lib().moonep_expert_ffn_w4q8, D, ctypes.byref(plan.desc), rp, H, I, _act(act), wp, sp, pitch, hp, yp,
         _stream(stream, D))
    return y, h


def moonep_expert_tile_w4(plan: Plan, H, I, rows_q8, product):
    """The tile that a product ("gate_up" or "down") of moonep_expert_ffn_w4, or with `rows_q8` of moonep_expert_ffn_w4q8, is
    computed in: weight rows and buffer rows."""
    if product not in PRODUCTS[:2]:
        raise MoonepError(f"product must be one of {PRODUCTS[:2]}, got {product!r}")
    tile = (ctypes.c_int32 * 2)()
    _check(lib().moonep_expert_tile_w4(ctypes.byref(plan.desc), H, I, int(bool(rows_q8)), PRODUCTS.index(product), tile))
    return tile[0], tile[1]


def _logits(logits, score):
    """Device pointer, type, rows, columns and the score's code of a router's logits."""
    kind = LOGITS.get(logits.dtype) if isinstance(logits, torch.Tensor) else None
    lp = _dev(logits, logits.dtype if kind is not None else torch.float32, "logits")
    if logits.dim() != 2:
        raise MoonepError("logits must be [T, E]")
    if score not in SCORES:
        raise MoonepError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    return lp, kind, logits.shape[0], logits.shape[1], SCORES[score]


@_on_its_stream
def moonep_router(logits, K, bias=None, score="softmax", groups=1, top_groups=1, normalize=True, scale=1.0,
                  ids=None, w=None, *, stream=None):
    """The K experts of each token and their weights, as moonep_plan takes them: (ids int32 [T, K], w fp32
    [T, K]) from logits fp32 or bf16 [T, E].  Experts are chosen by score + bias (fp32 [E]) among the
    top_groups best of `groups` groups; weights are the scores, divided by their sum with
    `normalize`, times `scale`."""
    lp, kind, T, E, code = _logits(logits, score)
    D = logits.device
    bp = None
    if bias is not None:
        bp = _dev(bias, torch.float32, "bias", D)
        if bias.numel() != E:
            raise MoonepError("bias must be [E]")
    ids, ip = _rows(ids, torch.int32, "ids", T, K, D, logits)
    w, wp = _rows(w, torch.float32, "w", T, K, D, logits)
    _run(lib().moonep_router, D, lp, kind, bp, T, E, K, code, groups, top_groups, int(bool(normalize)), scale, ip, wp,
         _stream(stream, D))
    return ids, w


@_on_its_stream
def moonep_router_bwd(logits, ids, g_w, score="softmax", normalize=True, scale=1.0, g_logits=None, *, stream=None):
    """The logits' gradient [T, E], of their type, from the weights' g_w fp32 [T, K] (moonep_combine_bwd's dw),
    for the ids int32 [T, K] that moonep_router chose."""
    lp, kind, T, E, code = _logits(logits, score)
    D = logits.device
    ip = _dev(ids, torch.int32, "ids", D)
    if ids.dim() != 2 or ids.shape[0] != T:
        raise MoonepError("ids must be [T, K]")
    K = ids.shape[1]
    gp = _rows(g_w, torch.float32, "g_w", T, K, D, logits)[1] if g_w is not None else None
    if gp is None:
        raise MoonepError("g_w must be a GPU tensor")
    g_logits, op = _rows(g_logits, logits.dtype, "g_logits", T, E, D, logits)
    _run(lib().moonep_router_bwd, D, lp, kind, ip, gp, T, E, K, code, int(bool(normalize)), scale, op,
         _stream(stream, D))
    return g_logits


def moonep_plan_status(plan: Plan, stream=None) -> dict:
    """Wait for the stream, then return the plan's statistics."""
    st = PlanStats()
    _check(lib().moonep_plan_status(ctypes.byref(plan.desc), ctypes.byref(st),
                                    _stream(stream, plan.blob.device)))
    return {n: getattr(st, n) for n, _ in PlanStats._fields_}
