"""MI355X-native expert-parallel dispatch planning for MoE layers.

A thin ctypes binding of the C ABI in include/moe_plan.h and
include/moe_experts.h (library load_balance_planning_amd/libmoe_plan.so, HIP
kernels for gfx950).  The
functions named like the C entry points only marshal arguments; every step of
the path runs in the library's kernels.  `Layer` is a convenience wrapper that
allocates the caller-owned buffers as torch tensors on the current HIP device
and runs the calls on torch's current stream -- PyTorch is used for device
memory and streams only.

There is no CPU fallback: the first call loads the HIP library (building it
in-tree with hipcc when none is there yet), and when it can be neither loaded
nor built that call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

from . import build as _build

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_HIP = -3
MOE_ERR_NONFINITE = -4
MOE_ERR_INTERNAL = -5
MOE_STATUS_NAN_LOGIT = 1
MOE_STATUS_PLAN_CHECK = 2
MOE_STATUS_BAD_TOPK = 4
MOE_STATUS_BAD_PAIRS = 8
MOE_STATUS_BAD_KEY = 16
MOE_STATUS_BAD_OMEGA = 32

_ERRORS = {MOE_ERR_INVALID_ARG: "invalid argument", MOE_ERR_UNSUPPORTED: "unsupported configuration",
           MOE_ERR_HIP: "HIP runtime error", MOE_ERR_NONFINITE: "non-finite gate logit",
           MOE_ERR_INTERNAL: "internal error"}


class MoePlanError(RuntimeError):
    def __init__(self, call: str, code: int):
        super().__init__("%s failed: %s (%d)" % (call, _ERRORS.get(code, "error"), code))
        self.code = code


class moe_plan_config(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("R", ctypes.c_int32),
                ("G", ctypes.c_int32), ("H", ctypes.c_int32), ("replica_budget", ctypes.c_int32),
                ("slots_per_rank", ctypes.c_int32), ("expert_bytes", ctypes.c_int64),
                ("token_bytes", ctypes.c_int64), ("max_refine_iters", ctypes.c_int32)]


class moe_plan_sizes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "topk", "omega", "experts", "pair", "inst_cap", "quota", "inst_offset",
        "rank_offset", "dispatch_elems", "n_slot", "expert_bytes", "token_bytes", "max_refine_iters",
        "workspace_bytes")]


class moe_route_out(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "topk_idx", "topk_val", "expert_count", "omega", "cooc", "trans")]


class moe_plan_out(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "n_inst", "inst_expert", "inst_rank", "inst_load", "rank_load", "quota", "slot_inst", "slot_rank")]


class moe_dispatch_out(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("perm", "slot_pos", "inst_offset", "rank_offset", "dispatch")]


class moe_place_out(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("expert_rank", "rank_experts", "intra", "n_swaps")]


class moe_predict_out(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("pred", "rank_tokens", "local")]


class moe_slot_out(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("slot_expert", "slot_main", "inst_slot")]


class moe_dedup_out(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "tok_ranks", "rank_rows", "rank_slots", "n_rows", "row_token", "row_slots", "rank_row_offset", "slot_row",
        "ddispatch")]


class moex_gate_config(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]


MOEX_SOFTMAX = 0
MOEX_SIGMOID = 1
BLOCK = 128  # columns (and, for matrices, rows) under one scale

EXPORTS = ("moe_plan_query", "moe_plan_create", "moe_plan_route", "moe_plan_hist", "moe_plan_plan",
           "moe_plan_dispatch", "moe_plan_step", "moe_plan_step_static", "moe_plan_combine", "moe_plan_place", "moe_plan_dedup_count",
           "moe_plan_dedup_dispatch", "moe_plan_quality", "moe_plan_predict", "moe_plan_slot_map",
           "moe_plan_replica_pull", "moe_plan_replica_push", "moe_plan_set_events", "moe_plan_set_gather_order",
           "moe_plan_device_info",
           "moe_plan_status", "moe_plan_destroy")
# include/moe_experts.h
EXPERT_EXPORTS = ("moex_gate", "moex_gate_grad", "moex_quantize", "moex_quantize_weights", "moex_swiglu",
                  "moex_swiglu_grad", "moex_matmul", "moex_wgrad", "moex_combine", "moex_combine_grad")

_LIB = None


def lib_path() -> str:
    return _build.LIB


def lib():
    """The loaded HIP library, built in-tree first when it is missing or was built from other
    sources than the ones in the tree (a hash of the sources is kept beside it)."""
    global _LIB
    if _LIB is None:
        if not _build.up_to_date():
            _build.build()
        l = ctypes.CDLL(_build.LIB)
        vp = ctypes.c_void_p
        l.moe_plan_query.argtypes = [vp, vp]
        l.moe_plan_create.argtypes = [vp, vp]
        l.moe_plan_route.argtypes = [vp, vp, vp, vp, vp]
        l.moe_plan_hist.argtypes = [vp, vp, vp, vp, vp]
        l.moe_plan_plan.argtypes = [vp, vp, vp, vp, vp]
        l.moe_plan_dispatch.argtypes = [vp, vp, vp, vp, vp]
        l.moe_plan_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp]
        l.moe_plan_step_static.argtypes = [vp] * 9
        l.moe_plan_combine.argtypes = [vp, vp, vp, vp, vp, vp]
        l.moe_plan_place.argtypes = [vp, vp, ctypes.c_int32, vp, vp]
        l.moe_plan_dedup_count.argtypes = [vp, vp, vp, ctypes.c_int32, vp, vp]
        l.moe_plan_dedup_dispatch.argtypes = [vp, vp, vp, ctypes.c_int32, vp, vp, vp]
        l.moe_plan_quality.argtypes = [vp, vp, vp, vp]
        l.moe_plan_predict.argtypes = [vp] * 8
        l.moe_plan_slot_map.argtypes = [vp, vp, vp, vp]
        l.moe_plan_device_info.argtypes = [ctypes.c_int, vp]
        l.moe_plan_set_events.argtypes = [vp, vp, vp]
        l.moe_plan_set_gather_order.argtypes = [vp, vp, vp]
        l.moe_plan_replica_pull.argtypes = [vp, vp, vp, ctypes.c_int64, vp, vp]
        l.moe_plan_replica_push.argtypes = [vp, vp, vp, ctypes.c_int64, vp, vp]
        l.moe_plan_status.argtypes = [vp, vp]
        l.moe_plan_destroy.argtypes = [vp]
        l.moe_plan_destroy.restype = None
        i32, i64 = ctypes.c_int32, ctypes.c_int64
        l.moex_gate.argtypes = [vp] * 8
        l.moex_gate_grad.argtypes = [vp] * 7
        l.moex_quantize.argtypes = [vp, vp, i64, i32, vp, vp, vp]
        l.moex_quantize_weights.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp, vp]
        l.moex_swiglu.argtypes = [vp, vp, i64, i32, vp, vp, vp]
        l.moex_swiglu_grad.argtypes = [vp, vp, vp, i64, i32, vp, vp, vp]
        l.moex_matmul.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, vp, vp]
        l.moex_wgrad.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, vp, vp]
        l.moex_combine.argtypes = [vp] * 6
        l.moex_combine_grad.argtypes = [vp] * 8
        for n in EXPORTS[:-1] + EXPERT_EXPORTS:
            getattr(l, n).restype = ctypes.c_int
        _LIB = l
    return _LIB


def _check(call: str, rc: int):
    if rc != MOE_OK:
        raise MoePlanError(call, rc)


# ---- entry points, same names as the C ABI ---------------------------------

def moe_plan_query(cfg: moe_plan_config) -> moe_plan_sizes:
    sz = moe_plan_sizes()
    _check("moe_plan_query", lib().moe_plan_query(ctypes.byref(cfg), ctypes.byref(sz)))
    return sz


def moe_plan_create(cfg: moe_plan_config) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check("moe_plan_create", lib().moe_plan_create(ctypes.byref(cfg), ctypes.byref(h)))
    return h


def moe_plan_route(h, logits: int, prev_topk: int | None, out: moe_route_out, stream: int):
    _check("moe_plan_route", lib().moe_plan_route(h, logits, prev_topk, ctypes.byref(out), stream))


def moe_plan_hist(h, topk_idx: int, prev_topk: int | None, out: moe_route_out, stream: int):
    _check("moe_plan_hist", lib().moe_plan_hist(h, topk_idx, prev_topk, ctypes.byref(out), stream))


def moe_plan_plan(h, omega: int, topk_idx: int | None, out: moe_plan_out, stream: int):
    _check("moe_plan_plan", lib().moe_plan_plan(h, omega, topk_idx, ctypes.byref(out), stream))


def moe_plan_dispatch(h, plan: moe_plan_out, hidden: int, out: moe_dispatch_out, stream: int):
    _check("moe_plan_dispatch", lib().moe_plan_dispatch(h, ctypes.byref(plan), hidden, ctypes.byref(out), stream))


def moe_plan_step(h, logits: int, prev_topk, hidden: int, route: moe_route_out, plan: moe_plan_out,
                  out: moe_dispatch_out, stream: int):
    _check("moe_plan_step", lib().moe_plan_step(h, logits, prev_topk, hidden, ctypes.byref(route), ctypes.byref(plan),
                                                ctypes.byref(out), stream))


def moe_plan_step_static(cfg: moe_plan_config, logits: int, prev_topk, hidden: int, route: moe_route_out,
                         plan: moe_plan_out, out: moe_dispatch_out, status: int, stream: int):
    _check("moe_plan_step_static", lib().moe_plan_step_static(ctypes.byref(cfg), logits, prev_topk, hidden,
                                                              ctypes.byref(route), ctypes.byref(plan),
                                                              ctypes.byref(out), status, stream))


def moe_plan_combine(h, topk_val: int, slot_pos: int, expert_out: int, out: int, stream: int):
    _check("moe_plan_combine", lib().moe_plan_combine(h, topk_val, slot_pos, expert_out, out, stream))


def moe_plan_place(h, cooc: int, max_swaps: int, out: moe_place_out, stream: int):
    _check("moe_plan_place", lib().moe_plan_place(h, cooc, max_swaps, ctypes.byref(out), stream))


def moe_plan_dedup_count(h, slot_key: int, key_rank, n_keys: int, out: moe_dedup_out, stream: int):
    _check("moe_plan_dedup_count", lib().moe_plan_dedup_count(h, slot_key, key_rank, n_keys, ctypes.byref(out), stream))


def moe_plan_dedup_dispatch(h, slot_key: int, key_rank, n_keys: int, hidden: int, out: moe_dedup_out, stream: int):
    _check("moe_plan_dedup_dispatch",
           lib().moe_plan_dedup_dispatch(h, slot_key, key_rank, n_keys, hidden, ctypes.byref(out), stream))


def moe_plan_quality(h, plan: moe_plan_out, out: int, stream: int):
    _check("moe_plan_quality", lib().moe_plan_quality(h, ctypes.byref(plan), out, stream))


def moe_plan_predict(h, topk_cur: int, trans: int, count_cur: int, key_rank, topk_next, out: moe_predict_out,
                     stream: int):
    _check("moe_plan_predict", lib().moe_plan_predict(h, topk_cur, trans, count_cur, key_rank, topk_next,
                                                      ctypes.byref(out), stream))


def moe_plan_slot_map(h, plan: moe_plan_out, out: moe_slot_out, stream: int):
    _check("moe_plan_slot_map", lib().moe_plan_slot_map(h, ctypes.byref(plan), ctypes.byref(out), stream))


def moe_plan_replica_pull(h, slot_expert: int, main_params: int, param_elems: int, replica_params: int, stream: int):
    _check("moe_plan_replica_pull",
           lib().moe_plan_replica_pull(h, slot_expert, main_params, param_elems, replica_params, stream))


def moe_plan_replica_push(h, slot_expert: int, replica_grads: int, param_elems: int, grad_accum: int, stream: int):
    _check("moe_plan_replica_push",
           lib().moe_plan_replica_push(h, slot_expert, replica_grads, param_elems, grad_accum, stream))


def moex_gate(h, gate: moex_gate_config, logits: int, bias, prev_topk, out: moe_route_out, weight: int, stream: int):
    _check("moex_gate", lib().moex_gate(h, ctypes.byref(gate), logits, bias, prev_topk, ctypes.byref(out), weight,
                                        stream))


def moex_gate_grad(h, gate: moex_gate_config, logits: int, topk_idx: int, grad_weight: int, grad_logits: int,
                   stream: int):
    _check("moex_gate_grad", lib().moex_gate_grad(h, ctypes.byref(gate), logits, topk_idx, grad_weight, grad_logits,
                                                  stream))


def moex_quantize(h, x: int, rows: int, cols: int, q: int, scale: int, stream: int):
    _check("moex_quantize", lib().moex_quantize(h, x, rows, cols, q, scale, stream))


def moex_quantize_weights(h, w: int, experts: int, n: int, k: int, q: int, scale: int, qt, scale_t, stream: int):
    _check("moex_quantize_weights",
           lib().moex_quantize_weights(h, w, experts, n, k, q, scale, qt, scale_t, stream))


def moex_swiglu(h, y: int, rows: int, f: int, q: int, scale: int, stream: int):
    _check("moex_swiglu", lib().moex_swiglu(h, y, rows, f, q, scale, stream))


def moex_swiglu_grad(h, y: int, grad: int, rows: int, f: int, q: int, scale: int, stream: int):
    _check("moex_swiglu_grad", lib().moex_swiglu_grad(h, y, grad, rows, f, q, scale, stream))


def moex_matmul(h, plan: moe_plan_out, inst_offset: int, x: int, x_scale: int, w: int, w_scale: int, n: int, k: int,
                y: int, stream: int):
    _check("moex_matmul", lib().moex_matmul(h, ctypes.byref(plan), inst_offset, x, x_scale, w, w_scale, n, k, y,
                                            stream))


def moex_wgrad(h, plan: moe_plan_out, inst_offset: int, dy: int, dy_scale: int, x: int, x_scale: int, n: int, k: int,
               dw: int, stream: int):
    _check("moex_wgrad", lib().moex_wgrad(h, ctypes.byref(plan), inst_offset, dy, dy_scale, x, x_scale, n, k, dw,
                                          stream))


def moex_combine(h, weight, slot_pos: int, expert_out: int, out: int, stream: int):
    _check("moex_combine", lib().moex_combine(h, weight, slot_pos, expert_out, out, stream))


def moex_combine_grad(h, weight: int, slot_pos: int, expert_out: int, grad_out: int, grad_expert_out: int,
                      grad_weight: int, stream: int):
    _check("moex_combine_grad", lib().moex_combine_grad(h, weight, slot_pos, expert_out, grad_out, grad_expert_out,
                                                        grad_weight, stream))


def moe_plan_set_events(h, gather_begin, gather_end):
    _check("moe_plan_set_events", lib().moe_plan_set_events(h, gather_begin, gather_end))


def moe_plan_set_gather_order(h, wait_event, done_event):
    _check("moe_plan_set_gather_order", lib().moe_plan_set_gather_order(h, wait_event, done_event))


def moe_plan_device_info(device: int = 0) -> dict:
    out = (ctypes.c_int64 * 6)()
    _check("moe_plan_device_info", lib().moe_plan_device_info(device, out))
    return dict(compute_units=out[0], clock_khz=out[1], memory_clock_khz=out[2], memory_bus_bits=out[3],
                l2_bytes=out[4], memory_bytes=out[5])


QUALITY_FIELDS = ("assignments", "same_rank", "same_node", "other_node", "replica_served", "max_rank_load",
                  "min_rank_load", "replicas")


def moe_plan_status(h) -> int:
    flags = ctypes.c_int32(0)
    _check("moe_plan_status", lib().moe_plan_status(h, ctypes.byref(flags)))
    return flags.value


def moe_plan_destroy(h):
    lib().moe_plan_destroy(h)


# ---- torch-owned buffers ----------------------------------------------------

def make_config(T, E, k, R, G, H, B, slots_per_rank=0, expert_bytes=-1, token_bytes=0,
                max_refine_iters=0) -> moe_plan_config:
    return moe_plan_config(T, E, k, R, G, H, B, slots_per_rank, expert_bytes, token_bytes, max_refine_iters)


def make_gate(score: str = "softmax", n_group: int = 1, topk_group: int = 1, group_top: int = 1, renorm: bool = True,
              scale: float = 1.0) -> moex_gate_config:
    """A router for Layer.gate: score "softmax" or "sigmoid", expert groups, weights renormalised and scaled."""
    kinds = {"softmax": MOEX_SOFTMAX, "sigmoid": MOEX_SIGMOID}
    if score not in kinds:
        raise ValueError("score must be one of %s" % sorted(kinds))
    return moex_gate_config(kinds[score], n_group, topk_group, group_top, int(bool(renorm)), scale)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


@dataclass
class RouteBuffers:
    topk_idx: object
    topk_val: object
    expert_count: object
    omega: object
    cooc: object
    trans: object

    def struct(self) -> moe_route_out:
        return moe_route_out(*(_ptr(getattr(self, n)) for n, _ in moe_route_out._fields_))


@dataclass
class PlanBuffers:
    n_inst: object
    inst_expert: object
    inst_rank: object
    inst_load: object
    rank_load: object
    quota: object
    slot_inst: object
    slot_rank: object

    def struct(self) -> moe_plan_out:
        return moe_plan_out(*(_ptr(getattr(self, n)) for n, _ in moe_plan_out._fields_))


@dataclass
class DispatchBuffers:
    perm: object
    slot_pos: object
    inst_offset: object
    rank_offset: object
    dispatch: object

    def struct(self) -> moe_dispatch_out:
        return moe_dispatch_out(*(_ptr(getattr(self, n)) for n, _ in moe_dispatch_out._fields_))


@dataclass
class PlaceBuffers:
    expert_rank: object
    rank_experts: object
    intra: object
    n_swaps: object

    def struct(self) -> moe_place_out:
        return moe_place_out(*(_ptr(getattr(self, n)) for n, _ in moe_place_out._fields_))


@dataclass
class DedupBuffers:
    tok_ranks: object
    rank_rows: object
    rank_slots: object
    n_rows: object = None
    row_token: object = None
    row_slots: object = None
    rank_row_offset: object = None
    slot_row: object = None
    ddispatch: object = None

    def struct(self) -> moe_dedup_out:
        return moe_dedup_out(*(_ptr(getattr(self, n)) for n, _ in moe_dedup_out._fields_))


def _addr(t):
    """Address of a tensor as ctypes takes it for a pointer argument (cheaper than an object of its own)."""
    return None if t is None else t.data_ptr()


def _current_stream(torch):
    """A function: the handle of torch's current stream on the device of an index.

    torch has it without the Python object around it (0.07 us a call, 1.15 through the public function, of the 7 to 9
    that a small call takes), under a private name, so a torch without that name goes through the public one."""
    return getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda index: torch.cuda.current_stream(index).cuda_stream)


@dataclass
class Blocks:
    """Quantized rows or matrices (include/moe_experts.h): q float8_e4m3fn [..., cols padded to 128], scale
    float8_e8m0fnu [..., blocks padded to 4] -- of rows one scale per 1 x 128, of matrices per 128 x 128."""
    q: object
    scale: object
    cols: int

    @staticmethod
    def padded(cols: int) -> int:
        return -(-cols // BLOCK) * BLOCK

    @staticmethod
    def scales(cols: int) -> int:
        return -(-(-(-cols // BLOCK)) // 4) * 4


class Layer:
    """One MoE layer's planner: a handle plus torch-allocated output buffers.

    route_out, plan_out and dispatch_out are one set of buffers, overwritten by the layer's next gate / route, plan
    and dispatch.  Calls that take them by default (gate_grad's topk_idx, the products' plan and inst_offset, the
    combines' slot_pos) are for the pass that ran last.  Where a layer runs forward several times before the first
    backward pass (micro-batches, pipelining, recomputation), keep copies of that pass's topk_idx, n_inst,
    inst_expert, inst_offset and slot_pos and pass them."""

    def __init__(self, cfg: moe_plan_config, device=None, cooc: bool = True, trans: bool = False,
                 topk_val: bool = True):
        import torch
        if not torch.cuda.is_available():
            raise RuntimeError("load_balance_planning_amd needs a HIP device")
        self.torch = torch
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.cfg = cfg
        self._index = self.device.index
        self._dims = (cfg.T, cfg.E, cfg.k, cfg.H)  # plain integers: a structure's fields cost more to read
        self._cap = cfg.E + cfg.replica_budget
        self._bf16 = torch.bfloat16
        self._current_stream = _current_stream(torch)
        self.sizes = moe_plan_query(cfg)
        with torch.cuda.device(self.device):
            self.handle = moe_plan_create(cfg)
        sz, dev, i32 = self.sizes, self.device, torch.int32
        T, E, k, R, H = cfg.T, cfg.E, cfg.k, cfg.R, cfg.H
        e = lambda n, dt=i32: torch.empty(int(n), dtype=dt, device=dev)
        self.route_out = RouteBuffers(
            topk_idx=e(sz.topk).view(T, k), topk_val=e(sz.topk, torch.float32).view(T, k) if topk_val else None,
            expert_count=e(E), omega=e(sz.omega).view(R, E),
            cooc=e(sz.pair).view(E, E) if cooc else None, trans=e(sz.pair).view(E, E) if trans else None)
        self.plan_out = PlanBuffers(
            n_inst=e(1), inst_expert=e(sz.inst_cap), inst_rank=e(sz.inst_cap), inst_load=e(sz.inst_cap),
            rank_load=e(R), quota=e(sz.quota).view(R, sz.inst_cap), slot_inst=e(sz.topk), slot_rank=e(sz.topk))
        self.dispatch_out = DispatchBuffers(
            perm=e(sz.topk), slot_pos=e(sz.topk), inst_offset=e(sz.inst_offset), rank_offset=e(sz.rank_offset),
            dispatch=e(sz.dispatch_elems, torch.int16).view(T * k, H))
        self._route_s = self.route_out.struct()
        self._plan_s = self.plan_out.struct()
        self._disp_s = self.dispatch_out.struct()
        self.place_out = None
        self.dedup_out = None

    def _stream(self, stream=None) -> int:
        if stream is None:
            return self._current_stream(self._index)
        if stream.device_index != self._index:
            raise ValueError("expected a stream of %s, got %s" % (self.device, stream))
        return stream.cuda_stream

    def route(self, logits, prev_topk=None, stream=None):
        self._check_tensor(logits, (self.cfg.T, self.cfg.E), self.torch.float32)
        if prev_topk is not None:
            self._check_tensor(prev_topk, (self.cfg.T, self.cfg.k), self.torch.int32)
        moe_plan_route(self.handle, _ptr(logits), _ptr(prev_topk), self._route_s, self._stream(stream))
        return self.route_out

    def hist(self, topk_idx, prev_topk=None, stream=None):
        """Histograms of a given top-k (moe_plan_hist); route_out.topk_idx is not touched."""
        self._check_tensor(topk_idx, (self.cfg.T, self.cfg.k), self.torch.int32)
        if prev_topk is not None:
            self._check_tensor(prev_topk, (self.cfg.T, self.cfg.k), self.torch.int32)
        moe_plan_hist(self.handle, _ptr(topk_idx), _ptr(prev_topk), self._route_s, self._stream(stream))
        return self.route_out

    def plan(self, omega=None, topk_idx=None, stream=None):
        """moe_plan_plan from a routing matrix [R][E] and the top-k [T][k] it counts; both default
        to this layer's route outputs."""
        omega = self.route_out.omega if omega is None else omega
        topk_idx = self.route_out.topk_idx if topk_idx is None else topk_idx
        self._check_tensor(omega, (self.cfg.R, self.cfg.E), self.torch.int32)
        self._check_tensor(topk_idx, (self.cfg.T, self.cfg.k), self.torch.int32)
        moe_plan_plan(self.handle, _ptr(omega), _ptr(topk_idx), self._plan_s, self._stream(stream))
        return self.plan_out

    def dispatch(self, hidden, stream=None):
        self._check_tensor(hidden, (self.cfg.T, self.cfg.H), None)
        if hidden.element_size() != 2:
            raise TypeError("hidden must be a 16-bit (bf16) tensor")
        moe_plan_dispatch(self.handle, self._plan_s, _ptr(hidden), self._disp_s, self._stream(stream))
        return self.dispatch_out

    def step(self, logits, hidden, prev_topk=None, stream=None):
        """route + plan + dispatch in one call (moe_plan_step)."""
        self._check_tensor(logits, (self.cfg.T, self.cfg.E), self.torch.float32)
        self._check_tensor(hidden, (self.cfg.T, self.cfg.H), None)
        if hidden.element_size() != 2:
            raise TypeError("hidden must be a 16-bit (bf16) tensor")
        if prev_topk is not None:
            self._check_tensor(prev_topk, (self.cfg.T, self.cfg.k), self.torch.int32)
        moe_plan_step(self.handle, _ptr(logits), _ptr(prev_topk), _ptr(hidden), self._route_s, self._plan_s,
                      self._disp_s, self._stream(stream))
        return self.route_out, self.plan_out, self.dispatch_out

    def combine(self, expert_out, out=None, stream=None):
        """Gate-weighted combine of expert outputs in dispatch order back to token order
        (moe_plan_combine), using this layer's topk_val and slot_pos."""
        T, k, H = self.cfg.T, self.cfg.k, self.cfg.H
        self._check_tensor(expert_out, (T * k, H), None)
        if expert_out.element_size() != 2:
            raise TypeError("expert_out must be a 16-bit (bf16) tensor")
        if self.route_out.topk_val is None:
            raise ValueError("combine needs the layer's topk_val buffer (create the Layer with topk_val=True)")
        if out is None:
            out = self.torch.empty((T, H), dtype=expert_out.dtype, device=self.device)
        self._check_tensor(out, (T, H), None)
        moe_plan_combine(self.handle, _ptr(self.route_out.topk_val), _ptr(self.dispatch_out.slot_pos),
                         _ptr(expert_out), _ptr(out), self._stream(stream))
        return out

    def gate(self, logits, gate: moex_gate_config, bias=None, prev_topk=None, stream=None, out=None):
        """Routing with scores, bias, groups and weights (moex_gate): (route_out, weight [T][k]).  The weights are the
        call's own (or in `out`), route_out is the layer's and overwritten by its next gate() or route()."""
        torch, (T, E, k, _) = self.torch, self._dims
        self._check_tensor(logits, (T, E), torch.float32)
        if bias is not None:
            self._check_tensor(bias, (E,), torch.float32)
        if prev_topk is not None:
            self._check_tensor(prev_topk, (T, k), torch.int32)
        weight = self._result(out, (T, k), torch.float32, stream)
        moex_gate(self.handle, gate, _addr(logits), _addr(bias), _addr(prev_topk), self._route_s, _addr(weight),
                  self._stream(stream))
        return self.route_out, weight

    def gate_grad(self, logits, gate: moex_gate_config, grad_weight, topk_idx=None, out=None, stream=None):
        """Gradient of gate()'s weights for the logits (moex_gate_grad).  topk_idx defaults to this layer's, which are
        those of its last gate() or route(): pass a copy if there was another since the one these weights came from."""
        torch, (T, E, k, _) = self.torch, self._dims
        topk_idx = self.route_out.topk_idx if topk_idx is None else topk_idx
        self._check_tensor(logits, (T, E), torch.float32)
        self._check_tensor(topk_idx, (T, k), torch.int32)
        self._check_tensor(grad_weight, (T, k), torch.float32)
        if out is None:
            out = self._empty((T, E), torch.float32, stream)
        else:
            self._check_tensor(out, (T, E), torch.float32)
        moex_gate_grad(self.handle, gate, _addr(logits), _addr(topk_idx), _addr(grad_weight), _addr(out),
                       self._stream(stream))
        return out

    def _empty(self, shape, dtype, stream):
        """A result of a call on `stream`, whose memory belongs to that stream: the allocator gives it to no other
        stream's tensors while the call may still write it."""
        if stream is None:
            return self.torch.empty(*shape, dtype=dtype, device=self.device)
        self._stream(stream)  # not one of another device
        with self.torch.cuda.stream(stream):
            return self.torch.empty(*shape, dtype=dtype, device=self.device)

    @staticmethod
    def _check_apart(out, t):
        """Rows that a kernel still reads may not be the ones it writes (contiguous tensors)."""
        a, b = out.data_ptr(), t.data_ptr()
        if a < b + t.numel() * t.element_size() and b < a + out.numel() * out.element_size():
            raise ValueError("out overlaps the rows that the call reads")

    def _result(self, out, shape, dtype, stream):
        """`out`, checked, or memory of the call's own."""
        if out is None:
            return self._empty(shape, dtype, stream)
        self._check_tensor(out, shape, dtype)
        return out

    def _result_blocks(self, out, stream, lead, cols, scale_lead=None) -> Blocks:
        if out is not None:
            if out.cols != cols:
                raise ValueError("out has %d columns, the result %d" % (out.cols, cols))
            self._check_blocks(out, lead, scale_lead)
            return out
        torch, scale_lead = self.torch, lead if scale_lead is None else scale_lead
        return Blocks(self._empty((*lead, Blocks.padded(cols)), torch.float8_e4m3fn, stream),
                      self._empty((*scale_lead, Blocks.scales(cols)), torch.float8_e8m0fnu, stream), cols)

    def _check_16bit(self, t, shape, name):
        """bf16, or its bit patterns in a 16-bit integer type."""
        self._check_tensor(t, shape, None)
        if t.dtype is not self._bf16 and (t.element_size() != 2 or t.dtype is self.torch.float16):
            raise TypeError("%s must be a bf16 tensor, not %s" % (name, t.dtype))

    def _check_blocks(self, b: Blocks, lead, scale_lead=None):
        torch = self.torch
        self._check_tensor(b.q, (*lead, Blocks.padded(b.cols)), torch.float8_e4m3fn)
        self._check_tensor(b.scale, (*(lead if scale_lead is None else scale_lead), Blocks.scales(b.cols)),
                           torch.float8_e8m0fnu)

    def quantize(self, x, stream=None, out=None) -> Blocks:
        """bf16 rows [n][cols] to Blocks of rows (moex_quantize), new ones or `out`."""
        if x.dim() != 2:
            raise ValueError("x must be [rows][cols]")
        rows, cols = x.shape
        self._check_16bit(x, (rows, cols), "x")
        out = self._result_blocks(out, stream, (rows,), cols)
        moex_quantize(self.handle, _addr(x), rows, cols, _addr(out.q), _addr(out.scale), self._stream(stream))
        return out

    def quantize_weights(self, w, transposed: bool = False, stream=None, out=None):
        """bf16 matrices [E][n][k] to Blocks of matrices (moex_quantize_weights); with transposed also those of the
        transposed matrices [E][k][n], from the same pass.  `out`: the Blocks to write (with transposed the pair), for
        instance those that a captured graph reads, after an optimizer step."""
        if w.dim() != 3:
            raise ValueError("w must be [experts][n][k]")
        E, n, k = w.shape
        self._check_16bit(w, (E, n, k), "w")
        blocks = lambda c: -(-c // BLOCK)
        out, out_t = (None, None) if out is None else out if transposed else (out, None)
        out = self._result_blocks(out, stream, (E, n), k, (E, blocks(n)))
        out_t = self._result_blocks(out_t, stream, (E, k), n, (E, blocks(k))) if transposed else Blocks(None, None, n)
        moex_quantize_weights(self.handle, _addr(w), E, n, k, _addr(out.q), _addr(out.scale), _addr(out_t.q),
                              _addr(out_t.scale), self._stream(stream))
        return (out, out_t) if transposed else out

    def swiglu(self, y, stream=None, out=None) -> Blocks:
        """silu(gate) * up of rows [n][2 f] (gate columns, then up), quantized (moex_swiglu), new Blocks or `out`."""
        if y.dim() != 2 or y.shape[1] % 2:
            raise ValueError("y must be [rows][2 f]")
        rows, f = y.shape[0], y.shape[1] // 2
        self._check_16bit(y, (rows, 2 * f), "y")
        out = self._result_blocks(out, stream, (rows,), f)
        moex_swiglu(self.handle, _addr(y), rows, f, _addr(out.q), _addr(out.scale), self._stream(stream))
        return out

    def swiglu_grad(self, y, grad, stream=None, out=None) -> Blocks:
        """Gradient of swiglu for y from grad [n][f], quantized (moex_swiglu_grad), new Blocks or `out`."""
        if y.dim() != 2 or y.shape[1] % 2:
            raise ValueError("y must be [rows][2 f]")
        rows, f = y.shape[0], y.shape[1] // 2
        self._check_16bit(y, (rows, 2 * f), "y")
        self._check_16bit(grad, (rows, f), "grad")
        out = self._result_blocks(out, stream, (rows,), 2 * f)
        moex_swiglu_grad(self.handle, _addr(y), _addr(grad), rows, f, _addr(out.q), _addr(out.scale),
                         self._stream(stream))
        return out

    def _product_plan(self, plan, inst_offset):
        """The struct of the instances a product runs over; by default this layer's plan and dispatch offsets, those of
        its last plan() and dispatch().  Of a given plan, n_inst and inst_expert are read."""
        inst_offset = self.dispatch_out.inst_offset if inst_offset is None else inst_offset
        cap = self._cap
        self._check_tensor(inst_offset, (cap + 1,), self.torch.int32)
        if plan is None:
            return self._plan_s, inst_offset
        self._check_tensor(plan.n_inst, (1,), self.torch.int32)
        self._check_tensor(plan.inst_expert, (cap,), self.torch.int32)
        s = moe_plan_out()  # the fields that the products read
        s.n_inst, s.inst_expert = plan.n_inst.data_ptr(), plan.inst_expert.data_ptr()
        return s, inst_offset

    def matmul(self, x: Blocks, w: Blocks, plan=None, inst_offset=None, out=None, stream=None):
        """Rows in dispatch order times their experts' matrices (moex_matmul): bf16 [T*k][n] of x, Blocks of rows
        [T*k][k], and w, Blocks of matrices [E][n][k]."""
        torch, (T, E, top, _) = self.torch, self._dims
        rows = T * top
        plan_s, inst_offset = self._product_plan(plan, inst_offset)
        n, k = w.q.shape[1], w.cols
        if x.cols != k:
            raise ValueError("x has %d columns, the matrices %d" % (x.cols, k))
        self._check_blocks(x, (rows,))
        self._check_blocks(w, (E, n), (E, -(-n // BLOCK)))
        if out is None:
            out = self._empty((rows, n), torch.bfloat16, stream)
        else:
            self._check_16bit(out, (rows, n), "out")
        moex_matmul(self.handle, plan_s, _addr(inst_offset), _addr(x.q), _addr(x.scale), _addr(w.q), _addr(w.scale), n, k,
                    _addr(out), self._stream(stream))
        return out

    def wgrad(self, dy: Blocks, x: Blocks, plan=None, inst_offset=None, out=None, stream=None):
        """Gradient of the experts' matrices (moex_wgrad): bf16 [E][n][k] of dy, Blocks of rows [T*k][n], and x,
        Blocks of rows [T*k][k]."""
        torch, (T, E, top, _) = self.torch, self._dims
        rows = T * top
        plan_s, inst_offset = self._product_plan(plan, inst_offset)
        self._check_blocks(dy, (rows,))
        self._check_blocks(x, (rows,))
        if out is None:
            out = self._empty((E, dy.cols, x.cols), torch.bfloat16, stream)
        else:
            self._check_16bit(out, (E, dy.cols, x.cols), "out")
        moex_wgrad(self.handle, plan_s, _addr(inst_offset), _addr(dy.q), _addr(dy.scale), _addr(x.q), _addr(x.scale),
                   dy.cols, x.cols, _addr(out), self._stream(stream))
        return out

    def _slot_positions(self, slot_pos):
        slot_pos = self.dispatch_out.slot_pos if slot_pos is None else slot_pos
        self._check_tensor(slot_pos, (self._dims[0] * self._dims[2],), self.torch.int32)
        return slot_pos

    def combine_weighted(self, expert_out, weight=None, slot_pos=None, out=None, stream=None):
        """Sum of each token's expert rows by the given weights [T][k] (moex_combine); without weights their plain
        sum, the gradient of the dispatch for its hidden rows."""
        torch, (T, _, k, H) = self.torch, self._dims
        slot_pos = self._slot_positions(slot_pos)
        self._check_16bit(expert_out, (T * k, H), "expert_out")
        if weight is not None:
            self._check_tensor(weight, (T, k), torch.float32)
        if out is None:
            out = self._empty((T, H), expert_out.dtype, stream)
        else:
            self._check_16bit(out, (T, H), "out")
            self._check_apart(out, expert_out)
        moex_combine(self.handle, _addr(weight), _addr(slot_pos), _addr(expert_out), _addr(out), self._stream(stream))
        return out

    def combine_grad(self, expert_out, grad_out, weight, slot_pos=None, stream=None, out=None):
        """Gradients of combine_weighted for the expert rows and the weights (moex_combine_grad):
        (grad_expert_out [T*k][H], grad_weight [T][k]), new ones or the pair `out`."""
        torch, (T, _, k, H) = self.torch, self._dims
        slot_pos = self._slot_positions(slot_pos)
        self._check_16bit(expert_out, (T * k, H), "expert_out")
        self._check_16bit(grad_out, (T, H), "grad_out")
        self._check_tensor(weight, (T, k), torch.float32)
        if out is None:
            grad_rows = self._empty((T * k, H), expert_out.dtype, stream)
            grad_weight = self._empty((T, k), torch.float32, stream)
        else:
            grad_rows, grad_weight = out
            self._check_16bit(grad_rows, (T * k, H), "out[0]")
            self._check_tensor(grad_weight, (T, k), torch.float32)
            self._check_apart(grad_rows, expert_out)
            self._check_apart(grad_rows, grad_out)
        moex_combine_grad(self.handle, _addr(weight), _addr(slot_pos), _addr(expert_out), _addr(grad_out),
                          _addr(grad_rows), _addr(grad_weight), self._stream(stream))
        return grad_rows, grad_weight

    def place(self, cooc=None, max_swaps: int = -1, stream=None):
        """Correlated expert placement from co-selection counts (moe_plan_place);
        cooc defaults to this layer's route_out.cooc."""
        torch, E, R = self.torch, self.cfg.E, self.cfg.R
        cooc = self.route_out.cooc if cooc is None else cooc
        if cooc is None:
            raise ValueError("place needs co-selection counts (create the Layer with cooc=True or pass cooc)")
        self._check_tensor(cooc, (E, E), torch.int32)
        if self.place_out is None:
            e = lambda n, dt=torch.int32: torch.empty(int(n), dtype=dt, device=self.device)
            self.place_out = PlaceBuffers(expert_rank=e(E), rank_experts=e(E).view(R, E // R),
                                          intra=e(1, torch.int64), n_swaps=e(1))
            self._place_s = self.place_out.struct()
        moe_plan_place(self.handle, _ptr(cooc), int(max_swaps), self._place_s, self._stream(stream))
        return self.place_out

    def _dedup_buffers(self, layout: bool):
        torch, T, k, R, H = self.torch, self.cfg.T, self.cfg.k, self.cfg.R, self.cfg.H
        e = lambda n, dt=torch.int32: torch.empty(int(n), dtype=dt, device=self.device)
        if self.dedup_out is None:
            self.dedup_out = DedupBuffers(tok_ranks=e(T), rank_rows=e(R * R).view(R, R), rank_slots=e(R * R).view(R, R))
        d = self.dedup_out
        if layout and d.ddispatch is None:
            d.n_rows, d.row_token, d.row_slots = e(1), e(T * k), e(T * k)
            d.rank_row_offset, d.slot_row = e(R + 1), e(T * k)
            d.ddispatch = e(T * k * H, torch.int16).view(T * k, H)
        self._dedup_s = d.struct()
        return d

    def _keys(self, slot_key, key_rank):
        T, k = self.cfg.T, self.cfg.k
        slot_key = self.route_out.topk_idx if slot_key is None else slot_key
        if tuple(slot_key.shape) not in ((T, k), (T * k,)) or not slot_key.is_contiguous() or \
                slot_key.dtype != self.torch.int32 or slot_key.device != self.device:
            raise ValueError("slot_key must be a contiguous int32 tensor of T*k keys on %s" % self.device)
        n = 0
        if key_rank is not None:
            if key_rank.dim() != 1 or not key_rank.is_contiguous() or key_rank.dtype != self.torch.int32 or \
                    key_rank.device != self.device:
                raise ValueError("key_rank must be a contiguous 1-d int32 tensor on %s" % self.device)
            n = key_rank.numel()
        return slot_key, key_rank, n

    def dedup_count(self, slot_key=None, key_rank=None, stream=None):
        """Deduplicated row counts (moe_plan_dedup_count).  slot_key defaults to
        this layer's top-k; key_rank None means the contiguous placement."""
        slot_key, key_rank, n = self._keys(slot_key, key_rank)
        self._dedup_buffers(False)
        moe_plan_dedup_count(self.handle, _ptr(slot_key), _ptr(key_rank), n, self._dedup_s, self._stream(stream))
        return self.dedup_out

    def dedup_dispatch(self, hidden, slot_key=None, key_rank=None, stream=None):
        """Deduplicated dispatch layout and row copy (moe_plan_dedup_dispatch)."""
        self._check_tensor(hidden, (self.cfg.T, self.cfg.H), None)
        if hidden.element_size() != 2:
            raise TypeError("hidden must be a 16-bit (bf16) tensor")
        slot_key, key_rank, n = self._keys(slot_key, key_rank)
        self._dedup_buffers(True)
        moe_plan_dedup_dispatch(self.handle, _ptr(slot_key), _ptr(key_rank), n, _ptr(hidden), self._dedup_s,
                                self._stream(stream))
        return self.dedup_out

    def quality(self, stream=None):
        """Plan-quality counters of this layer's plan (moe_plan_quality): an int64 tensor of 8
        on the device, in QUALITY_FIELDS order."""
        if getattr(self, "_quality", None) is None:
            self._quality = self.torch.empty(8, dtype=self.torch.int64, device=self.device)
        moe_plan_quality(self.handle, self._plan_s, _ptr(self._quality), self._stream(stream))
        return self._quality

    def predict(self, topk_cur, trans, count_cur, key_rank=None, topk_next=None, stream=None):
        """Token-shuffle prediction (moe_plan_predict): returns (pred [T], rank_tokens [R], local [2])
        device tensors; local counts next-layer slots on the predicted / source rank when
        topk_next is given."""
        torch, T, E, k, R = self.torch, self.cfg.T, self.cfg.E, self.cfg.k, self.cfg.R
        self._check_tensor(topk_cur, (T, k), torch.int32)
        self._check_tensor(trans, (E, E), torch.int32)
        self._check_tensor(count_cur, (E,), torch.int32)
        if key_rank is not None:
            self._check_tensor(key_rank, (E,), torch.int32)
        if topk_next is not None:
            self._check_tensor(topk_next, (T, k), torch.int32)
        if getattr(self, "_pred", None) is None:
            self._pred = (torch.empty(T, dtype=torch.int32, device=self.device),
                          torch.empty(R, dtype=torch.int32, device=self.device),
                          torch.empty(2, dtype=torch.int64, device=self.device))
        out = moe_predict_out(*(_ptr(x) for x in self._pred))
        moe_plan_predict(self.handle, _ptr(topk_cur), _ptr(trans), _ptr(count_cur), _ptr(key_rank), _ptr(topk_next),
                         out, self._stream(stream))
        return self._pred

    def slot_map(self, stream=None):
        """Replica slot map of this layer's plan (moe_plan_slot_map): (slot_expert [R][N_slot],
        slot_main [R][N_slot], inst_slot [E+B]) device tensors."""
        torch, R = self.torch, self.cfg.R
        ns, cap = int(self.sizes.n_slot), int(self.sizes.inst_cap)
        if getattr(self, "_slots", None) is None:
            e = lambda n: torch.empty(n, dtype=torch.int32, device=self.device)
            self._slots = (e(R * ns).view(R, ns), e(R * ns).view(R, ns), e(cap))
        moe_plan_slot_map(self.handle, self._plan_s, moe_slot_out(*(_ptr(x) for x in self._slots)),
                          self._stream(stream))
        return self._slots

    def replica_pull(self, main_params, replica_params, stream=None):
        """moe_plan_replica_pull with this layer's slot map: main_params [E][P] -> replica_params
        [R][N_slot][P] (16-bit tensors)."""
        E, R, ns = self.cfg.E, self.cfg.R, int(self.sizes.n_slot)
        P = main_params.shape[-1]
        self._check_tensor(main_params, (E, P), None)
        self._check_tensor(replica_params, (R, ns, P), None)
        moe_plan_replica_pull(self.handle, _ptr(self._slots[0]), _ptr(main_params), int(P), _ptr(replica_params),
                              self._stream(stream))
        return replica_params

    def replica_push(self, replica_grads, grad_accum, stream=None):
        """moe_plan_replica_push with this layer's slot map: replica_grads [R][N_slot][P] ->
        grad_accum [R][R][E/R][P]."""
        E, R, ns = self.cfg.E, self.cfg.R, int(self.sizes.n_slot)
        P = replica_grads.shape[-1]
        self._check_tensor(replica_grads, (R, ns, P), None)
        self._check_tensor(grad_accum, (R, R, E // R, P), None)
        moe_plan_replica_push(self.handle, _ptr(self._slots[0]), _ptr(replica_grads), int(P), _ptr(grad_accum),
                              self._stream(stream))
        return grad_accum

    def time_gather(self, begin=None, end=None):
        """Record two torch.cuda.Events around the gather kernel of every later dispatch / step
        call of this layer (moe_plan_set_events); with no events, stop.  The events must have
        been recorded once already (torch creates the HIP event on its first record)."""
        if begin is None:
            moe_plan_set_events(self.handle, None, None)
        else:
            moe_plan_set_events(self.handle, ctypes.c_void_p(begin.cuda_event), ctypes.c_void_p(end.cuda_event))

    def order_gather(self, wait=None, done=None):
        """moe_plan_set_gather_order with torch.cuda.Events (each None for none): this layer's
        row copies wait for `wait` and record `done`.  The events must have been recorded once
        already (torch creates the HIP event on its first record)."""
        ptr = lambda ev: None if ev is None else ctypes.c_void_p(ev.cuda_event)
        moe_plan_set_gather_order(self.handle, ptr(wait), ptr(done))

    def status(self) -> int:
        return moe_plan_status(self.handle)

    def _check_tensor(self, t, shape, dtype):
        if t.shape != shape or t.get_device() != self._index or not t.is_contiguous():
            raise ValueError("expected a contiguous %s tensor of shape %s on %s" % (dtype, shape, self.device))
        if dtype is not None and t.dtype != dtype:
            raise TypeError("expected dtype %s, got %s" % (dtype, t.dtype))

    def close(self):
        if getattr(self, "handle", None) is not None:
            moe_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
