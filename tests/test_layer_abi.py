"""Host-side validation of the layer operators' C entry points: bad arguments are refused with a
status and a text before anything reaches the GPU (no compute here)."""
import ctypes
import os

import pytest

from gated_delta_rule_70_amd import binding

needs_lib = pytest.mark.skipif(not os.path.exists(binding.LIB_PATH),
                               reason="libgdr.so not built (run __graft_entry__.build())")
pytestmark = needs_lib
A = 1 << 24  # 16-byte aligned addresses, far apart, never dereferenced

SCAN = ("x", "a", "b", "A_log", "dt_bias")
CALLS = {
    "scan_fwd": (SCAN + ("h0", "cu", "out", "hT", "states", "ws", "wsb"), binding.ScanDims,
                 dict(B=2, T=100, D=16, num_seqs=0, dtype=1, flags=0), dict(cu=None), "gdr_channel_scan_fwd"),
    "scan_bwd": (SCAN + ("states", "cu", "dout", "dhT", "dx", "da", "db", "dA_log", "ddt_bias", "dh0", "ws", "wsb"),
                 binding.ScanDims, dict(B=2, T=100, D=16, num_seqs=0, dtype=1, flags=0), dict(cu=None),
                 "gdr_channel_scan_bwd"),
    "scan_step": (SCAN + ("state_in", "state_out", "out"), binding.ScanDims,
                  dict(B=2, T=1, D=16, num_seqs=0, dtype=1, flags=0), {}, "gdr_channel_scan_step"),
    "ffn_fwd": (("x", "w_gate", "w_up", "h", "gate", "up"), binding.FfnDims, dict(M=8, D=16, F=24, dtype=1, act=0), {},
                "gdr_gated_ffn_fwd"),
    "ffn_bwd": (("x", "w_gate", "w_up", "gate", "up", "dh", "dx", "dw_gate", "dw_up", "ws", "wsb"), binding.FfnDims,
                dict(M=8, D=16, F=24, dtype=1, act=0), {}, "gdr_gated_ffn_bwd"),
    "ce_fwd": (("x", "w", "targets", "loss", "lse", "ws", "wsb"), binding.CeDims,
               dict(N=8, D=16, V=50, dtype=1, flags=0), {}, "gdr_linear_ce_fwd"),
    "ce_bwd": (("x", "w", "targets", "lse", "dloss", "dx", "dw", "ws", "wsb"), binding.CeDims,
               dict(N=8, D=16, V=50, dtype=1, flags=0), {}, "gdr_linear_ce_bwd"),
}


def call(which, over):
    names, struct, dims, ptrs, entry = CALLS[which]
    dims = dict(dims)
    at = {n: A * (i + 1) for i, n in enumerate(names)}
    at["wsb"] = 1 << 23
    at.update(ptrs)
    no_dims = over.get("dims", 1) is None
    for k, v in over.items():
        if k in dims:
            dims[k] = v
        elif k != "dims":
            assert k in at, k
            at[k] = v
    d = struct(*[dims[f[0]] for f in struct._fields_])
    args = [ctypes.c_int64(at[n]) if n == "wsb" else (None if at[n] is None else ctypes.c_void_p(at[n])) for n in names]
    lib = binding.load()
    st = getattr(lib, entry)(*args, None if no_dims else ctypes.byref(d), None)
    return binding.STATUS[st], lib.gdr_last_error().decode()


REJECTS = [
    ("scan_fwd", dict(dims=None), "NULL", "dims"),
    ("scan_fwd", dict(dtype=5), "DTYPE", "dtype"),
    ("scan_fwd", dict(flags=1), "FLAGS", "flags"),
    ("scan_fwd", dict(D=0), "DIMS", "D"),
    ("scan_fwd", dict(T=-1), "DIMS", "T"),
    ("scan_fwd", dict(T=1 << 31), "DIMS", "T"),
    ("scan_fwd", dict(B=1 << 40, D=1 << 30), "DIMS", "overflow"),
    ("scan_fwd", dict(B=1 << 31), "DIMS", "too many"),
    ("scan_fwd", dict(cu=A * 50), "DIMS", "B == 1"),
    ("scan_fwd", dict(cu=A * 50, B=1), "DIMS", "num_seqs"),
    ("scan_fwd", dict(cu=A * 50 + 2, B=1, num_seqs=2), "ALIGN", "cu_seqlens"),
    ("scan_fwd", dict(cu=A * 8, B=1, num_seqs=2), "ALIAS", "out overlaps cu_seqlens"),
    ("scan_fwd", dict(x=None), "NULL", "x"),
    ("scan_fwd", dict(A_log=None), "NULL", "A_log"),
    ("scan_fwd", dict(out=None), "NULL", "out"),
    ("scan_fwd", dict(b=A * 3 + 8), "ALIGN", "b is"),
    ("scan_fwd", dict(out=A + 32), "ALIAS", "out overlaps x"),
    ("scan_fwd", dict(hT=A * 6 + 16), "ALIAS", "hT overlaps h0"),
    ("scan_fwd", dict(states=A * 9), "ALIAS", "hT overlaps states"),
    ("scan_bwd", dict(states=None), "NULL", "states"),
    ("scan_bwd", dict(dA_log=None), "NULL", "dA_log"),
    ("scan_bwd", dict(wsb=3), "DIMS", "workspace_bytes"),
    ("scan_bwd", dict(ws=None), "NULL", "workspace"),
    ("scan_bwd", dict(dx=A * 8), "ALIAS", "dx overlaps dout"),
    ("scan_bwd", dict(da=A * 10), "ALIAS", "overlaps"),
    ("scan_bwd", dict(ws=A * 16 + 4), "ALIGN", "workspace"),
    ("scan_step", dict(T=2), "DIMS", "T must be 1"),
    ("scan_step", dict(flags=2), "FLAGS", "step"),
    ("scan_step", dict(state_in=None), "NULL", "state_in"),
    ("scan_step", dict(state_out=A * 6 + 16), "ALIAS", "state_out overlaps state_in"),
    ("ffn_fwd", dict(act=2), "FLAGS", "act"),
    ("ffn_fwd", dict(M=-1), "DIMS", "M"),
    ("ffn_fwd", dict(D=(1 << 20) + 1), "DIMS", "D"),
    ("ffn_fwd", dict(M=(1 << 31) - 1, F=1 << 20), "DIMS", "too large"),
    ("ffn_fwd", dict(gate=None), "NULL", "together"),
    ("ffn_fwd", dict(w_up=None), "NULL", "w_up"),
    ("ffn_fwd", dict(h=A * 2), "ALIAS", "h overlaps w_gate"),
    ("ffn_fwd", dict(up=A * 5 + 16), "ALIAS", "gate overlaps up"),
    ("ffn_bwd", dict(wsb=10), "DIMS", "workspace_bytes"),
    ("ffn_bwd", dict(dh=None), "NULL", "dh"),
    ("ffn_bwd", dict(dx=A), "ALIAS", "dx overlaps x"),
    ("ffn_bwd", dict(dw_up=A * 8 + 64), "ALIAS", "dw_gate overlaps dw_up"),
    ("ce_fwd", dict(flags=1), "FLAGS", "flags"),
    ("ce_fwd", dict(V=0), "DIMS", "V"),
    ("ce_fwd", dict(N=(1 << 31) - 1, V=(1 << 31) - 1), "DIMS", "too large"),
    ("ce_fwd", dict(targets=None), "NULL", "targets"),
    ("ce_fwd", dict(lse=A * 4), "ALIAS", "loss overlaps lse"),
    ("ce_fwd", dict(wsb=1), "DIMS", "workspace_bytes"),
    ("ce_bwd", dict(lse=None), "NULL", "lse"),
    ("ce_bwd", dict(dw=A * 2), "ALIAS", "dw overlaps w"),
    ("ce_bwd", dict(targets=A * 3 + 4), "ALIGN", "targets"),
]


@pytest.mark.parametrize("which,over,status,text", REJECTS, ids=["%s:%s" % (r[0], "-".join(r[1])) for r in REJECTS])
def test_rejects(which, over, status, text):
    got, msg = call(which, over)
    assert got == "GDR_ERR_" + status and text in msg, (got, msg)


def test_sizes_of_buffers():
    lib = binding.load()
    d = binding.ScanDims(2, 513, 8, 0, 1, 0)
    assert lib.gdr_channel_scan_states_elems(ctypes.byref(d), 0) == 2 * 3 * 8
    d = binding.ScanDims(1, 513, 8, 4, 1, 0)
    assert lib.gdr_channel_scan_states_elems(ctypes.byref(d), 1) == (513 // 256 + 5) * 8
    for f in (lib.gdr_channel_scan_states_elems, lib.gdr_channel_scan_fwd_workspace_bytes, lib.gdr_channel_scan_bwd_workspace_bytes):
        assert f(ctypes.byref(binding.ScanDims(2, 4, 0, 0, 1, 0)), 0) == -1
    assert lib.gdr_gated_ffn_bwd_workspace_bytes(ctypes.byref(binding.FfnDims(1, 1, 1, 9, 0))) == -1
    for f in (lib.gdr_linear_ce_fwd_workspace_bytes, lib.gdr_linear_ce_bwd_workspace_bytes):
        assert f(ctypes.byref(binding.CeDims(1, 1, 0, 0, 0))) == -1
        assert f(ctypes.byref(binding.CeDims(100, 64, 5000, 1, 0))) > 0


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("T", [0, 1, 256, 257, 300, 100000])
def test_sizes_of_an_empty_batch(T, dtype):
    lib = binding.load()
    d = binding.ScanDims(0, T, 20, 0, dtype, 0)
    for f in (lib.gdr_channel_scan_states_elems, lib.gdr_channel_scan_fwd_workspace_bytes, lib.gdr_channel_scan_bwd_workspace_bytes):
        assert f(ctypes.byref(d), 0) == 0


def test_type_of_the_kept_projections():
    """With gate and up in fp32 each is twice as long as bf16 ones, and the activation is still checked."""
    at = A * 5 + 8 * 24 * 2
    got, msg = call("ffn_fwd", dict(act=256, up=at))
    assert got == "GDR_ERR_ALIAS" and "gate overlaps up" in msg
    got, msg = call("ffn_bwd", dict(act=256, dx=A * 4 + 8 * 24 * 2))
    assert got == "GDR_ERR_ALIAS" and "dx overlaps gate" in msg
    for act in (257 + 1, 512, -1):
        got, msg = call("ffn_fwd", dict(act=act))
        assert got == "GDR_ERR_FLAGS" and "act" in msg
