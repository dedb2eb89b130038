"""How far a NaN reaches in windowed attention: rows that see it are NaN, rows of tiles that never meet it are bit for bit
what they were (rows of a tile that holds it without seeing it are computed again, within the bounds of the definition:
test_gpu_seq_window.py)."""
import pytest
import torch

from layer_ref import visible
from test_gpu_seq_window import BF, F32, setup
import sparse_graph_attention_csr_gb300 as sga

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("H,D", [(2, 64), (3, 128), (1, 32)])
def test_nan_in_one_row(H, D, dt, causal):
    lens, window, sinks, col = [300, 90, 420, 200], 50, 2, 3
    T, tile = sum(lens), 128 if dt == BF else 64
    plan, ptr, Q, K, V, dO = setup(lens, H, 1, D, dt, causal, window, sinks)
    vis = torch.block_diag(*[visible(n, causal, window, sinks).float() for n in lens]).bool()   # row i sees key j
    at = torch.arange(T, device="cuda") // tile
    n = int(at[-1]) + 1
    meet = torch.zeros(n, n, dtype=torch.bool, device="cuda")   # tiles with a visible pair: those that are walked
    i, j = vis.nonzero(as_tuple=True)
    meet[at[i], at[j]] = True

    def run(rows=None):
        out, lse = sga.seq_attn_fwd(plan, Q, K, V)
        # (rows that were computed again without having seen the NaN are rounded elsewhere: the backward is given what they were)
        back = out if rows is None else torch.where(rows[:, None, None], out, clean["out"])
        dQ, dK, dV = sga.seq_attn_bwd(plan, Q, K, V, back, lse, dO)
        return {"out": out, "lse": lse[..., None], "dQ": dQ, "dK": dK, "dV": dV}

    clean, columns = run(), torch.arange(D, device="cuda")
    for what in ("K", "V", "Q", "dO"):
        t = {"K": K, "V": V, "Q": Q, "dO": dO}[what]
        for row in (1, 150, 301, 500, 809, 1009):
            own = torch.arange(T, device="cuda") == row
            rows = vis[:, row] if what in "KV" else own                  # queries that meet the NaN
            was = t[row, 0, col].clone()
            t[row, 0, col] = torch.nan
            got = run(rows)
            t[row, 0, col] = was
            assert plan.device_error() == 0
            keys = vis[rows].any(0)                                      # and the keys that these see
            far_rows = ~meet[at, at[row]] if what in "KV" else ~own
            far_keys = ~meet[at[rows]].any(0)[at]
            assert far_keys.any() and far_rows.any()
            one, every, none = columns == col, columns >= 0, columns < 0
            # (rows that are NaN, in which columns; rows that stay bit for bit; the columns that stay so in every row)
            expect = {"K": {"out": (rows, every, far_rows, none), "lse": (rows, every, ~rows, none), "dQ": (rows, every, far_rows, none),
                            "dK": (keys, every, far_keys, none), "dV": (keys, every, far_keys, none)},
                      "V": {"out": (rows, one, far_rows, ~one), "lse": (rows, none, far_rows, every), "dQ": (rows, every, far_rows, none),
                            "dK": (keys, every, far_keys, none), "dV": (keys, none, far_keys, every)},
                      "Q": {"out": (rows, every, ~own, none), "lse": (rows, every, ~own, none), "dQ": (rows, every, ~own, none),
                            "dK": (keys, every, far_keys, none), "dV": (keys, every, far_keys, none)},
                      "dO": {"out": (rows, none, far_rows, every), "lse": (rows, none, far_rows, every), "dQ": (rows, every, ~own, none),
                             "dK": (keys, every, far_keys, none), "dV": (keys, one, far_keys, ~one)}}[what]
            for name, (hit, where, far, stay) in expect.items():
                a, b = clean[name], got[name]
                where, stay = where[:a.shape[-1]], stay[:a.shape[-1]]
                shared = a.shape[1] == 1 or what in "KV"                  # (a query head's NaN stays in that head's rows)
                heads = slice(None) if shared else slice(0, 1)
                assert torch.isnan(b[hit][:, heads][..., where]).all(), (what, row, name)
                assert torch.equal(a[far], b[far]) and torch.equal(a[..., stay], b[..., stay]), (what, row, name)
                if not shared:
                    assert torch.equal(a[:, 1:], b[:, 1:]), (what, row, name)
