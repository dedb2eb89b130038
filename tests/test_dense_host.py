"""Host-side refusals of packed-sequence attention, layer norm and embedding:
checked before any device call (CPU only)."""
import ctypes

import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)


def test_host_tensors_and_dtypes_are_refused():
    sp = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sga.SeqPlan(sp, 1, 32)
    with pytest.raises(TypeError):
        sga.SeqPlan(sp, 1, 32, torch.float16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sga.layer_norm_fwd(torch.zeros(2, 4))
    with pytest.raises(ValueError, match="CUDA tensor"):
        sga.embed_fwd(torch.zeros(2, dtype=torch.int64), torch.zeros(3, 4))
    with pytest.raises(ValueError, match="CUDA tensor"):
        sga.embed_bwd(torch.zeros(2, dtype=torch.int64), torch.zeros(2, 4), 3)


def test_sequence_plan_arguments():
    lib = sga.load_library()
    out = ctypes.c_void_p()
    new = lambda ptr, B, H, Hk, D, dt=1, causal=1, o=ctypes.byref(out): lib.sga_seq_plan_create(ptr, B, H, Hk, D, dt, causal, None, o)
    assert new(P, 4, 2, 2, 48) == sga.SGA_EUNSUPPORTED
    assert new(P, 4, 3, 2, 64) == sga.SGA_EUNSUPPORTED
    assert new(P, 4, 256, 256, 128) == sga.SGA_EUNSUPPORTED
    assert new(P, 4, 2, 2, 64, dt=2) == sga.SGA_EUNSUPPORTED
    assert new(P, -1, 2, 2, 64) == sga.SGA_EINVAL
    assert new(None, 4, 2, 2, 64) == sga.SGA_EINVAL
    assert new(ODD, 4, 2, 2, 64) == sga.SGA_EINVAL
    assert new(P, 4, 2, 2, 64, causal=2) == sga.SGA_EINVAL
    assert new(P, 4, 2, 2, 64, o=None) == sga.SGA_EINVAL
    assert lib.seq_attn_fwd(None, P, P, P, 4, 1.0, P, P, None) == sga.SGA_EINVAL
    assert lib.seq_attn_bwd(None, P, P, P, P, P, P, 4, 1.0, P, P, P, P, 0, None) == sga.SGA_EINVAL
    assert lib.sga_seq_plan_rows(None) == 0 and lib.sga_seq_bwd_workspace_bytes(None) == 0
    code = ctypes.c_int32()
    assert lib.sga_seq_read_device_error(None, None, ctypes.byref(code)) == sga.SGA_EINVAL
    lib.sga_seq_plan_destroy(None)


def test_layer_norm_arguments():
    lib = sga.load_library()
    fwd = lambda X=P, w=P, b=P, N=4, C=8, eps=1e-5, dt=0, wdt=0, o=P: lib.layer_norm_fwd(X, w, b, N, C, eps, dt, wdt, o, P, P, None)
    assert fwd(N=-1) == sga.SGA_EINVAL and fwd(C=0) == sga.SGA_EINVAL
    assert fwd(C=(1 << 20) + 1) == sga.SGA_EUNSUPPORTED
    assert fwd(dt=2) == sga.SGA_EUNSUPPORTED and fwd(wdt=1) == sga.SGA_EUNSUPPORTED
    assert fwd(w=None) == sga.SGA_EINVAL
    assert fwd(eps=-1.0) == sga.SGA_EINVAL and fwd(eps=float("nan")) == sga.SGA_EINVAL
    assert fwd(X=None) == sga.SGA_EINVAL and fwd(X=ODD) == sga.SGA_EINVAL and fwd(w=ODD) == sga.SGA_EINVAL
    assert fwd(N=0) == sga.SGA_OK
    bwd = lambda w=P, dX=P, dw=P, db=P, ws=P, n=1 << 40: lib.layer_norm_bwd(P, w, P, P, P, 4, 8, 0, 0, dX, dw, db, ws, n, None)
    assert bwd(w=None) == sga.SGA_EINVAL and bwd(dX=None) == sga.SGA_EINVAL
    assert bwd(dw=None) == sga.SGA_EINVAL and bwd(ws=None) == sga.SGA_EINVAL
    assert bwd(n=0) == sga.SGA_EWORKSPACE


def test_embedding_arguments():
    lib = sga.load_library()
    fwd = lambda ids=P, b=4, t=P, N=4, V=5, C=8, dt=0, o=P: lib.embed_fwd(ids, b, t, N, V, C, 1.0, dt, o, None)
    assert fwd(b=2) == sga.SGA_EINVAL and fwd(N=-1) == sga.SGA_EINVAL and fwd(V=-1) == sga.SGA_EINVAL
    assert fwd(C=0) == sga.SGA_EINVAL and fwd(dt=3) == sga.SGA_EUNSUPPORTED
    assert fwd(N=1 << 31) == sga.SGA_EUNSUPPORTED and fwd(V=1 << 31) == sga.SGA_EUNSUPPORTED
    assert fwd(ids=None) == sga.SGA_EINVAL and fwd(t=None) == sga.SGA_EINVAL and fwd(o=ODD) == sga.SGA_EINVAL
    assert fwd(ids=ctypes.c_void_p(4100), b=8) == sga.SGA_EINVAL
    assert fwd(N=0) == sga.SGA_OK
    bwd = lambda d=P, t=P, ws=P, n=1 << 40: lib.embed_bwd(P, 4, d, 4, 5, 8, 1.0, -1, 0, t, ws, n, None)
    assert bwd(d=None) == sga.SGA_EINVAL and bwd(t=None) == sga.SGA_EINVAL and bwd(ws=None) == sga.SGA_EINVAL
    assert bwd(n=0) == sga.SGA_EWORKSPACE
    assert lib.sga_embed_bwd_workspace_bytes(0, 5, 8) == 0
    assert lib.sga_embed_read_device_error(None, None) == sga.SGA_EINVAL
