"""The plain form of windowed attention among the measured cases against the definition in 64 bits (CPU): it is what the
kernels' outputs are compared with there."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT
from layer_ref import window_reference, within


def measured():
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,window,sinks", [
    ([300, 50], 1, 200), ([300, 50], 60, 190), ([100, 300, 50], 40, 120),   # first rows that lie behind what the windows reach
    ([127, 1, 129], 3, 200), ([1, 1, 260], 2, 1), ([40], 5, 100), ([500], 17, 0), ([256, 3], 300, 130)])
def test_windowed_attention(lens, window, sinks, causal):
    m, H, Hk, D = measured(), 2, 1, 32
    T, g = sum(lens), torch.Generator().manual_seed(1)
    ptr = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)
    n = lambda h: torch.randn(T, h, D, generator=g)
    st = {"seq_ptr": ptr, "reach": min(window, max(lens)), "window": window, "sinks": sinks, "causal": causal, "kv_heads": Hk, "dim": D,
          "Q": n(H), "K": n(Hk), "V": n(Hk), "dOut": n(H)}
    st["out"], st["lse"] = m._win_fwd(st)
    got = dict(zip(("out", "lse", "dQ", "dK", "dV"), (st["out"], st["lse"], *m._win_bwd(st))))
    for name, t in window_reference(ptr, st["Q"], st["K"], st["V"], D ** -0.5, causal, window, sinks, st["dOut"], st["out"]).items():
        within(got[name], t, name)
