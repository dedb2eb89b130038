"""Layer norm of more rows than its grids have groups, at widths of every path."""
import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga
from dense_ref import norm_reference, within

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("dt,wt", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("C", [63, 513, 520, 1000, 1025, 2048, 4095, 4096, 4097, 8200])
def test_rows_beyond_the_grid(C, dt, wt):
    """A block (of a row at these widths) takes several rows one after the other:
    more than 32 an SM in the forward, 8 in its widest form, 4 in the backward."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    N = (33 if C <= 4096 else 9) * sms + 5
    g = torch.Generator(device="cuda").manual_seed(C)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    X, dO = (n(N, C) * 1.7 + 0.3).to(DT[dt]), n(N, C).to(DT[dt])
    w, b = (n(C) * 0.2 + 1).to(DT[wt]), (n(C) * 0.2).to(DT[wt])
    ref = norm_reference(X, w, b, 1e-5, dO)
    out, mean, rstd = sga.layer_norm_fwd(X, w, b)
    dX, dw, db = sga.layer_norm_bwd(X, w, mean, rstd, dO)
    for name, t in {"out": out, "mean": mean, "rstd": rstd, "dX": dX, "dweight": dw, "dbias": db}.items():
        within(t, ref[name], name)
    again = sga.layer_norm_bwd(X, w, mean, rstd, dO)
    assert all(torch.equal(a, c) for a, c in zip(again, (dX, dw, db)))
