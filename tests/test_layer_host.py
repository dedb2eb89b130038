"""Host-side refusals of the transformer-layer operators: checked before any device call (CPU only)."""
import ctypes

import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)


def test_rotary_arguments():
    for bad in (dict(D=48), dict(D=64, dims=72), dict(D=64, dims=24), dict(D=64, dims=-16), dict(D=64, base=0.0), dict(D=64, base=float("inf")),
                dict(D=32, freqs=[1.0] * 15), dict(D=32, freqs=[float("nan")] * 16), dict(D=32, sections=[8, 7]),
                dict(D=32, sections=[4, 4, 4, 2, 2]), dict(D=32, sections=[17, -1]), dict(D=32, sections=[])):
        with pytest.raises(ValueError):
            sga.Rotary(**bad)
    r = sga.Rotary(64, 32, sections=[4, 12])
    assert (r.axes, r.dims, len(r.freqs)) == (2, 32, 16) and r.freqs[0] == 1.0 and abs(r.freqs[8] - 0.01) < 1e-15
    assert sga.Rotary(32, 0).freqs == []


def test_rotary_table():
    class Table(ctypes.Structure):
        _fields_ = [("D", ctypes.c_int32), ("rot", ctypes.c_int32), ("axes", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                    ("turn", ctypes.c_uint64 * 64), ("axis", ctypes.c_uint8 * 64)]

    lib, t = sga.load_library(), Table()
    f = (ctypes.c_double * 8)(2 * 3.141592653589793, 3.141592653589793, -3.141592653589793 / 2, 1.0, 0.0, -1e-300, 1e300, 0.5)
    sec = (ctypes.c_int32 * 2)(3, 5)
    new = lambda D=32, rot=16, freqs=f, s=sec, axes=2, inter=1, o=ctypes.byref(t): lib.sga_rotary_init(o, D, rot, freqs, s, axes, inter)
    assert new() == sga.SGA_OK
    assert list(t.axis[:8]) == [0, 0, 0, 1, 1, 1, 1, 1] and (t.D, t.rot, t.axes, t.interleaved) == (32, 16, 2, 1)
    assert t.turn[0] == 0 and t.turn[1] == 1 << 63 and t.turn[2] == 3 << 62 and t.turn[4] == 0
    assert abs(t.turn[3] / 2 ** 64 - 0.15915494309189535) < 1e-16
    assert t.turn[5] == 0    # (just under a whole turn)
    assert new(D=48) == sga.SGA_EUNSUPPORTED
    assert new(o=None) == new(rot=8) == new(rot=48) == new(freqs=None) == new(axes=0) == new(axes=5) == new(s=None) == new(inter=2) == sga.SGA_EINVAL
    assert new(s=(ctypes.c_int32 * 2)(3, 6)) == new(s=(ctypes.c_int32 * 2)(3, 4)) == new(s=(ctypes.c_int32 * 2)(9, -1)) == sga.SGA_EINVAL
    assert new(freqs=(ctypes.c_double * 8)(float("inf"))) == sga.SGA_EINVAL
    assert new() == sga.SGA_OK
    R = ctypes.byref(t)
    fwd = lambda r=R, Q=P, ldq=64, K=P, ldk=32, pos=P, pb=8, wq=P, wk=P, T=4, H=2, Hk=1, eps=1e-6, dt=0, wdt=0, o=P, rq=P, rk=P: \
        lib.qk_norm_rope_fwd(r, Q, ldq, K, ldk, pos, pb, wq, wk, T, H, Hk, eps, dt, wdt, o, P, rq, rk, None)
    assert fwd(T=0) == sga.SGA_OK
    for bad in (dict(r=None), dict(Q=None), dict(Q=ODD), dict(ldq=63), dict(ldq=66), dict(ldk=30), dict(pos=None), dict(pos=ODD), dict(pb=2),
                dict(wq=None), dict(wq=ODD), dict(T=-1), dict(H=0), dict(Hk=0), dict(eps=-1.0), dict(eps=float("nan")), dict(o=None), dict(rq=None),
                dict(rq=None, rk=None)):
        assert fwd(**bad) == sga.SGA_EINVAL, bad
    for bad in (dict(dt=2), dict(wdt=1), dict(H=1024, ldq=32768, Hk=1)):
        assert fwd(**bad) == sga.SGA_EUNSUPPORTED, bad
    bwd = lambda wq=P, wk=P, rq=P, rk=P, dq=P, dwq=P, dwk=P, ws=P, n=1 << 40, dQ=P: \
        lib.qk_norm_rope_bwd(R, P, 64, P, 32, P, 8, wq, wk, rq, rk, dq, P, 4, 2, 1, 0, 0, dQ, P, dwq, dwk, ws, n, None)
    for bad in (dict(wq=None), dict(rq=None), dict(rq=None, rk=None), dict(dq=None), dict(dQ=None), dict(dwq=None), dict(dwq=ODD), dict(ws=None),
                dict(ws=ODD), dict(wq=None, wk=None)):
        assert bwd(**bad) == sga.SGA_EINVAL, bad
    assert bwd(n=0) == sga.SGA_EWORKSPACE
    t.axis[7] = 2
    assert fwd() == sga.SGA_EINVAL


def test_host_tensors_are_refused():
    rot, x = sga.Rotary(32), torch.zeros(2, 1, 32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sga.qk_norm_rope_fwd(rot, x, x, torch.arange(2))
    with pytest.raises(ValueError, match="CUDA tensor"):
        sga.qk_norm_rope_bwd(rot, x, x, torch.arange(2), None, None, None, None, x, x)


def test_windowed_plan_arguments():
    lib, out = sga.load_library(), ctypes.c_void_p()
    new = lambda window, sinks, causal=1, D=64, ptr=P: lib.sga_seq_plan_create_windowed(ptr, 4, 2, 2, D, 1, causal, window, sinks, None, ctypes.byref(out))
    assert new(-1, 0) == new(0, 1) == new(4, -1) == new(4, 1, causal=2) == new(4, 1, ptr=None) == sga.SGA_EINVAL
    assert new(4, 1, D=48) == sga.SGA_EUNSUPPORTED
    sp = torch.tensor([0, 4], dtype=torch.int32)
    for window, sinks in ((0, 0), (-3, 0), (None, 2), (4, -1)):
        with pytest.raises(ValueError, match="window|sinks"):
            sga.SeqPlan(sp, 1, 32, window=window, sinks=sinks)


def test_gated_ff_arguments():
    lib = sga.load_library()
    fwd = lambda X=P, T=4, F=16, M=24, act=0, dt=1, o=P, G=P, U=P, ws=P, n=1 << 40: \
        lib.gated_ff_fwd(X, P, P, T, F, M, act, dt, o, G, U, ws, n, None)
    assert fwd(T=0) == sga.SGA_OK
    for bad in (dict(X=None), dict(X=ODD), dict(T=-1), dict(F=0), dict(M=0), dict(act=3), dict(act=-1), dict(o=None), dict(o=ODD), dict(G=None),
                dict(U=None), dict(G=ODD), dict(F=15, ws=None), dict(F=15, ws=ODD)):
        assert fwd(**bad) == sga.SGA_EINVAL, bad
    for bad in (dict(dt=2), dict(T=1 << 31), dict(F=(1 << 20) + 1), dict(M=(1 << 20) + 1), dict(T=(1 << 31) - 2000, M=1 << 20)):
        assert fwd(**bad) == sga.SGA_EUNSUPPORTED, bad
    assert fwd(F=15, n=0) == fwd(dt=0, n=0) == sga.SGA_EWORKSPACE
    bwd = lambda G=P, dt=1, dX=P, dWg=P, dWu=P, ws=P, n=1 << 40, act=0: lib.gated_ff_bwd(P, P, P, G, P, P, 4, 16, 24, act, dt, dX, dWg, dWu, ws, n, None)
    for bad in (dict(G=None), dict(G=ODD), dict(dX=ODD), dict(dWg=None), dict(dWu=None), dict(dWu=ODD), dict(ws=None), dict(ws=ODD), dict(act=9)):
        assert bwd(**bad) == sga.SGA_EINVAL, bad
    assert bwd(n=0) == sga.SGA_EWORKSPACE
    assert bwd(dX=None, dWg=None, dWu=None) == sga.SGA_OK
    assert lib.sga_gated_ff_fwd_workspace_bytes(0, 16, 24, 1) == lib.sga_gated_ff_bwd_workspace_bytes(4, 0, 24, 1) == 0
    assert lib.sga_gated_ff_bwd_workspace_bytes(4, 16, 24, 0) >= 4 * 24 * 2 * 6
    assert lib.sga_gated_ff_read_device_error(None, None) == sga.SGA_EINVAL
    with pytest.raises(ValueError, match="CUDA tensor"):
        sga.gated_ff_fwd(torch.zeros(2, 16), torch.zeros(16, 8), torch.zeros(16, 8))
