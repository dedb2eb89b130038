"""The dense operators on arrays of more than 2^31 elements: the last rows are
what the same call gives on them alone."""
import pytest
import torch

import sparse_graph_attention_csr_gb300 as sga

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB")
    yield
    torch.cuda.empty_cache()


def filled(*shape, seed=0):
    t = torch.empty(*shape, device="cuda", dtype=torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for i in range(0, shape[0], 1 << 18):
        t[i:i + (1 << 18)].normal_(generator=g)
    return t


def test_packed_sequences():
    n, T, H, D = 100, 1 << 20, 17, 128   # 2^31.09 elements of Q
    lens = [n] * (T // n) + [T % n]
    ptr = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
    plan = sga.SeqPlan(ptr, H, D, causal=True)
    Q, K, V, dO = (filled(T, H, D, seed=s) for s in range(4))
    assert Q.numel() > 1 << 31
    out, lse = sga.seq_attn_fwd(plan, Q, K, V)
    grads = sga.seq_attn_bwd(plan, Q, K, V, out, lse, dO)
    tail = 25 * 128   # whole row tiles, whole sequences: the same tiles as alone
    first = T - tail
    while first % 128 or first % n:
        first -= 1
    small = sga.SeqPlan((ptr[ptr >= first] - first).contiguous(), H, D, causal=True)
    x = [t[first:].clone() for t in (Q, K, V, dO)]
    o, l = sga.seq_attn_fwd(small, *x[:3])
    for a, b in zip((out, lse, *grads), (o, l, *sga.seq_attn_bwd(small, *x[:3], o, l, x[3]))):
        assert torch.equal(a[first:], b)
    assert plan.device_error() == 0


@pytest.mark.parametrize("C", [512, 513])
def test_layer_norm(C):
    N = (1 << 31) // C + 5000
    X, dO, w = filled(N, C), filled(N, C, seed=1), torch.rand(C, device="cuda") + 0.5
    assert X.numel() > 1 << 31
    out, mean, rstd = sga.layer_norm_fwd(X, w, w)
    dX, dw, db = sga.layer_norm_bwd(X, w, mean, rstd, dO)
    s = slice(N - 1000, None)
    o, m, r = sga.layer_norm_fwd(X[s].clone(), w, w)
    assert torch.equal(out[s], o) and torch.equal(mean[s], m) and torch.equal(rstd[s], r)
    assert torch.equal(dX[s], sga.layer_norm_bwd(X[s].clone(), w, m, r, dO[s].clone())[0])
    # db is the columns' sums of dO, summed in parts that fp32 holds well
    want = sum(dO[i:i + (1 << 18)].double().sum(0) for i in range(0, N, 1 << 18))
    mag = sum(dO[i:i + (1 << 18)].double().abs().sum(0) for i in range(0, N, 1 << 18))
    assert ((db.double() - want).abs() <= (N / 600 + 600) * 2 ** -24 * mag).all()   # (a block's rows, then the blocks)


def test_embedding():
    C, V = 512, 50000
    N = (1 << 31) // C + 5000
    g = torch.Generator(device="cuda").manual_seed(0)
    ids = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    table = filled(V, C)
    out = sga.embed_fwd(ids, table)
    assert out.numel() > 1 << 31
    for i in range(0, N, 1 << 18):
        assert torch.equal(out[i:i + (1 << 18)], table[ids[i:i + (1 << 18)].long()])
    out.fill_(1)
    dT = sga.embed_bwd(ids, out, V)
    assert torch.equal(dT, torch.bincount(ids, minlength=V)[:, None].expand(V, C).bfloat16())
    few = sga.embed_bwd(ids % 3, out, 300)
    assert torch.equal(few[:3], torch.bincount(ids % 3)[:, None].expand(3, C).float().bfloat16()) and (few[3:] == 0).all()


def test_a_table_past_2_31_elements():
    C, V, N = 1024, (1 << 21) + 1000, 5000
    ids = torch.randint(V - 2000, V, (N,), device="cuda")
    table = torch.zeros(V, C, device="cuda", dtype=torch.bfloat16)
    table[V - 2000:] = filled(2000, C)
    assert torch.equal(sga.embed_fwd(ids, table), table[ids])
    dO = filled(N, C, seed=1)
    dT = sga.embed_bwd(ids, dO, V)
    assert dT.numel() > 1 << 31
    assert torch.equal(dT[V - 2000:], sga.embed_bwd(ids - (V - 2000), dO, 2000)) and not dT[:V - 2000].any()
