"""The C-ABI library builds, loads and exports every declared symbol (CPU only)."""

import ctypes
import os
import re

import pytest

import table_embedding_bags_gb300 as tbe
from table_embedding_bags_gb300.build import INCLUDE, build

HEADER = os.path.join(INCLUDE, "tbe.h")


def declared_functions():
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = re.findall(r"\b(tbe_[a-z_0-9]+)\s*\(", src)
    return sorted(set(names))


@pytest.fixture(scope="module")
def lib():
    build()
    return tbe.load_library()


def test_header_matches_binding_list():
    assert declared_functions() == sorted(tbe.EXPORTED)


def test_every_declared_symbol_is_exported(lib):
    for name in declared_functions():
        assert hasattr(lib, name), name
        assert ctypes.cast(getattr(lib, name), ctypes.c_void_p).value


def test_host_only_calls(lib):
    assert lib.tbe_plan_device_bytes(1) == 256
    assert lib.tbe_plan_device_bytes(0) == 0
    assert lib.tbe_plan_device_bytes(tbe.TBE_MAX_TABLES + 1) == 0
    assert lib.tbe_status_string(tbe.TBE_ERR_WORKSPACE) == b"workspace too small"
    assert b"sm_103a" in lib.tbe_version()
    t = tbe.get_tuning()
    assert t["long_run_threshold"] >= 1 and t["fwd_unroll"] in (4, 8)
    with pytest.raises(tbe.TBEError):
        tbe.set_tuning(fwd_unroll=3)
    with pytest.raises(tbe.TBEError):
        tbe.set_tuning(long_chunk=33)
    assert tbe.get_tuning() == t


@pytest.mark.parametrize("field,bad", [("fwd_lanes_per_row", 3), ("fwd_lanes_per_row", 64), ("fwd_lanes_per_row", 0),
                                       ("red_unroll", 6), ("fwd_ring", 4), ("short_item_lookups", 31),
                                       ("fwd_blocks_per_sm", -1), ("long_run_threshold", 0)])
def test_tuning_rejects_out_of_range(lib, field, bad):
    t = tbe.get_tuning()
    with pytest.raises(tbe.TBEError):
        tbe.set_tuning(**{field: bad})
    assert tbe.get_tuning() == t  # a rejected call changes nothing


def test_tuning_round_trip(lib):
    t = tbe.get_tuning()
    assert t["long_chunk"] == 0 and t["fwd_ring"] == 3 and t["red_unroll"] in (4, 8)
    try:
        tbe.set_tuning(long_chunk=128, short_item_lookups=64, fwd_lanes_per_row=8, red_unroll=8, fwd_ring=0)
        u = tbe.get_tuning()
        assert (u["long_chunk"], u["short_item_lookups"], u["fwd_lanes_per_row"], u["red_unroll"], u["fwd_ring"]) == \
            (128, 64, 8, 8, 0)
    finally:
        tbe.set_tuning(**t)
    assert tbe.get_tuning() == t
    # null arguments are rejected on the host before any CUDA call
    assert lib.tbe_plan_create(None, None, 0, None, None) == tbe.TBE_ERR_INVALID_ARG
    assert lib.tbe_forward(None, None, None, 0, None, 0, None, None, None, None) == tbe.TBE_ERR_INVALID_ARG
    assert lib.tbe_backward_workspace_bytes(None, 1, 1) == 0
    # the bounded-wait self-test checks its arguments before any CUDA call
    assert lib.tbe_wait_selftest(2, 10, None, None) == tbe.TBE_ERR_INVALID_ARG
    assert lib.tbe_wait_selftest(0, 0, None, None) == tbe.TBE_ERR_INVALID_ARG


def test_exact_update_rejects_without_plan(lib):
    opt = tbe.Optimizer(tbe.TBE_OPT_EXACT_SGD, 0.1, 0.0)
    rc = lib.tbe_exact_update(None, ctypes.byref(opt), None, None, None, 0, None, 0, None, None, None)
    assert rc == tbe.TBE_ERR_INVALID_ARG
    rc = lib.tbe_exact_update(None, None, None, None, None, 0, None, 0, None, None, None)
    assert rc == tbe.TBE_ERR_INVALID_ARG


def _layout(T, trb, doff, woff, wdt, out_dtype=0, pooling=0):
    import numpy as np

    keep = [np.ascontiguousarray(trb, np.int64), np.ascontiguousarray(doff, np.int32),
            np.ascontiguousarray(woff, np.int64), np.ascontiguousarray(wdt, np.int32)]
    L = tbe._Layout(T, *(a.ctypes.data for a in keep), None, out_dtype, pooling)
    return L, keep


# layouts that tbe_plan_create must refuse before it touches the device
BAD_LAYOUTS = {
    "no_tables": (dict(T=0, trb=[0], doff=[0], woff=[], wdt=[]), tbe.TBE_ERR_INVALID_ARG),
    "too_many_tables": (dict(T=tbe.TBE_MAX_TABLES + 1, trb=[0, 1], doff=[0, 4], woff=[0], wdt=[0]),
                        tbe.TBE_ERR_INVALID_ARG),
    "row_base_not_zero": (dict(T=1, trb=[5, 10], doff=[0, 4], woff=[0], wdt=[0]), tbe.TBE_ERR_INVALID_ARG),
    "rows_decrease": (dict(T=2, trb=[0, 10, 4], doff=[0, 4, 8], woff=[0, 256], wdt=[0, 0]),
                      tbe.TBE_ERR_INVALID_ARG),
    "zero_width": (dict(T=2, trb=[0, 10, 20], doff=[0, 4, 4], woff=[0, 256], wdt=[0, 0]), tbe.TBE_ERR_INVALID_ARG),
    "unknown_dtype": (dict(T=1, trb=[0, 10], doff=[0, 4], woff=[0], wdt=[7]), tbe.TBE_ERR_INVALID_ARG),
    "unknown_out_dtype": (dict(T=1, trb=[0, 10], doff=[0, 4], woff=[0], wdt=[0], out_dtype=9),
                          tbe.TBE_ERR_INVALID_ARG),
    "unknown_pooling": (dict(T=1, trb=[0, 10], doff=[0, 4], woff=[0], wdt=[0], pooling=2), tbe.TBE_ERR_INVALID_ARG),
    "row_not_16_bytes": (dict(T=1, trb=[0, 10], doff=[0, 3], woff=[0], wdt=[0]), tbe.TBE_ERR_UNSUPPORTED),
    "half_row_not_16_bytes": (dict(T=1, trb=[0, 10], doff=[0, 4], woff=[0], wdt=[1]), tbe.TBE_ERR_UNSUPPORTED),
    "table_not_aligned": (dict(T=2, trb=[0, 10, 20], doff=[0, 4, 8], woff=[0, 8], wdt=[0, 0]),
                          tbe.TBE_ERR_UNSUPPORTED),
    "rows_beyond_int32": (dict(T=1, trb=[0, 1 << 31], doff=[0, 4], woff=[0], wdt=[0]), tbe.TBE_ERR_UNSUPPORTED),
}


@pytest.mark.parametrize("name", sorted(BAD_LAYOUTS))
def test_plan_create_refuses_bad_layouts(lib, name):
    kw, want = BAD_LAYOUTS[name]
    L, _keep = _layout(kw["T"], kw["trb"], kw["doff"], kw["woff"], kw["wdt"], kw.get("out_dtype", 0), kw.get("pooling", 0))
    meta = (ctypes.c_uint8 * (1 << 20))()
    base = (ctypes.addressof(meta) + 15) // 16 * 16
    h = ctypes.c_void_p()
    rc = lib.tbe_plan_create(ctypes.byref(L), ctypes.c_void_p(base), (1 << 20) - 16, None, ctypes.byref(h))
    assert rc == want and not h.value


def test_plan_create_checks_its_metadata_buffer(lib):
    L, _keep = _layout(1, [0, 10], [0, 4], [0], [0])
    meta = (ctypes.c_uint8 * 4096)()
    base = (ctypes.addressof(meta) + 15) // 16 * 16
    h = ctypes.c_void_p()
    need = lib.tbe_plan_device_bytes(1)
    assert lib.tbe_plan_create(ctypes.byref(L), None, need, None, ctypes.byref(h)) == tbe.TBE_ERR_INVALID_ARG
    assert lib.tbe_plan_create(ctypes.byref(L), ctypes.c_void_p(base), need - 1, None,
                               ctypes.byref(h)) == tbe.TBE_ERR_INVALID_ARG
    assert lib.tbe_plan_create(ctypes.byref(L), ctypes.c_void_p(base + 4), need, None,
                               ctypes.byref(h)) == tbe.TBE_ERR_INVALID_ARG


def test_argument_checks_before_the_abi():
    """The binding's tensor checks (no GPU needed: host tensors are refused
    first, then dtype and size)."""
    import torch

    import table_embedding_bags_gb300 as tbe

    with pytest.raises(tbe.TBEError, match="CUDA"):
        tbe._need(torch.zeros(4, dtype=torch.int64), (torch.int64,), 4, "indices")
    with pytest.raises(tbe.TBEError, match="required"):
        tbe._need(None, (torch.int64,), 4, "indices")
    tbe._need(None, (torch.float32,), 4, "per_sample_weights", optional=True)


class _ScanInputs(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("sequences", ctypes.c_int32), ("channels", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("offsets_i32", ctypes.c_int32), ("x", ctypes.c_void_p),
                ("recur", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("x_stride", ctypes.c_int64),
                ("recur_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64), ("decay", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("h0", ctypes.c_void_p), ("sharpness", ctypes.c_float)]


class _ScanGrads(ctypes.Structure):
    _fields_ = [("dx", ctypes.c_void_p), ("drecur", ctypes.c_void_p), ("dgate", ctypes.c_void_p),
                ("dx_stride", ctypes.c_int64), ("drecur_stride", ctypes.c_int64), ("dgate_stride", ctypes.c_int64),
                ("ddecay", ctypes.c_void_p), ("dh0", ctypes.c_void_p)]


def test_states_in_place_are_refused(lib):
    """A sequence's last state may be written before another block has read its first one: h0 and h_last (dh_last and
    dh0) must not overlap.  Host memory stands in for the device's; a misaligned h (dh), refused in another way, keeps
    every call from launching anything."""
    N, S, C = 64, 2, 8
    room = (ctypes.c_float * 8192)()
    base = (ctypes.addressof(room) + 255) // 256 * 256
    x, decay, offsets, states, h0, far = (base + 4096 * i for i in range(6))
    size = 4 * S * C
    a = _ScanInputs(N, S, C, tbe.TBE_F32, 0, x, x, x, C, C, C, decay, offsets, h0, 8.0)
    b = _ScanInputs(N, S, C, tbe.TBE_F32, 0, x, x, x, C, C, C, decay, offsets, None, 8.0)
    for where, rc in ((h0, tbe.TBE_ERR_INVALID_ARG), (h0 + size - 4, tbe.TBE_ERR_INVALID_ARG),
                      (h0 - size + 4, tbe.TBE_ERR_INVALID_ARG), (h0 + size, tbe.TBE_ERR_UNSUPPORTED),
                      (h0 - size, tbe.TBE_ERR_UNSUPPORTED), (far, tbe.TBE_ERR_UNSUPPORTED)):
        assert lib.tbe_gated_scan(ctypes.byref(a), x + 1, C, where, states, None, 0, None, None) == rc
        g = _ScanGrads(x, x, x, C, C, C, decay, where)
        assert lib.tbe_gated_scan_backward(ctypes.byref(b), x + 1, C, h0, states, ctypes.byref(g), None, 0, None,
                                           None) == rc
    assert lib.tbe_gated_scan(ctypes.byref(b), x + 1, C, h0, states, None, 0, None, None) == tbe.TBE_ERR_UNSUPPORTED
    g = _ScanGrads(x, x, x, C, C, C, decay, None)
    assert lib.tbe_gated_scan_backward(ctypes.byref(b), x + 1, C, h0, states, ctypes.byref(g), None, 0, None,
                                       None) == tbe.TBE_ERR_UNSUPPORTED


def test_binding_is_built_again_for_another_pytorch(monkeypatch):
    """The compiled binding uses PyTorch's C++ interface and Python's: one built against others is not reused."""
    import sys

    import torch

    from table_embedding_bags_gb300 import build as b

    b.build()
    built = []
    monkeypatch.setattr(b, "_compile_marshal", lambda verbose: built.append(1))
    b.build()
    assert not built
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    b.build()
    assert built == [1]
    monkeypatch.undo()
    monkeypatch.setattr(b, "_compile_marshal", lambda verbose: built.append(1))
    monkeypatch.setattr(sys, "version", "2.7")
    b.build()
    assert built == [1, 1]


def test_the_package_needs_pytorch_only_where_tensors_are():
    """Loading the library and its host-only calls work where PyTorch cannot be imported (and do not wait for it)."""
    import subprocess
    import sys

    code = """
import sys
class Block:
    def find_spec(self, name, path=None, target=None):
        if name.split(".")[0] == "torch":
            raise ImportError("torch")
sys.meta_path.insert(0, Block())
import table_embedding_bags_gb300 as tbe
assert tbe.load_library().tbe_plan_device_bytes(1) == 256 and "sm_103a" in tbe.version()
assert tbe.TBE_SCAN_STEP == 8 and tbe.TBE_ADAMW_BLOCK == 256
assert "tbe_gated_scan" in dir(tbe) and not hasattr(tbe, "no_such_name")
from table_embedding_bags_gb300 import build
assert build.build() == build.LIB
try:
    tbe.tbe_gated_scan
except ImportError:
    print("ok")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(tbe.__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.stdout.strip() == "ok", r.stderr
    from table_embedding_bags_gb300 import AdamWPlan, tbe_adamw_step, tbe_gated_scan, training

    assert tbe.tbe_gated_scan is tbe_gated_scan is training.tbe_gated_scan
    assert tbe.AdamWPlan is AdamWPlan and tbe.tbe_adamw_step is tbe_adamw_step
