"""GPU attention over a store that appends have filled: held to the 64-bit attention of what the oracle's appends leave, and
element by element to that of the values themselves."""
import numpy as np
import pytest
import torch

import q8_bounds as B
import varlen_gqa_attention_gb300 as pkg
from oracle import sdpa_varlen_oracle as O
from oracle import step_oracle as S
from test_q8_attention_gpu import run_q8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


@pytest.fixture(params=["auto", "splitk", "prefill"])
def route(request):
    pkg.set_route_policy({"auto": pkg.ROUTE_AUTO, "splitk": pkg.ROUTE_SPLITK, "prefill": pkg.ROUTE_PREFILL}[request.param])
    yield request.param
    pkg.set_route_policy(pkg.ROUTE_AUTO)


def test_a_store_that_append_has_filled(dev, route):
    """A prompt, then tokens one by one.  The attention is that of what the oracle's append leaves, to the roundings; and from
    that of the values themselves each element is at most as far as the weighted errors of the stored values and twice
    the largest error of the row's scores allow."""
    Hq, Hkv, D, rows, n = 4, 2, 128, 128, 100
    g = torch.Generator().manual_seed(17)
    q, k, v = (torch.randn(n, h, D, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    stored = pkg.q8_store(rows, 1, Hkv, D, device=dev)
    parts = [t.numpy() for t in pkg.q8_store(rows, 1, Hkv, D)]
    table = torch.tensor([1.0, 0.0]).expand(rows, D // 2, 2).contiguous()  # no rotation
    tabled = table.to(dev)
    for a, b in [(0, 70)] + [(t, t + 1) for t in range(70, n)]:
        seq = np.array([[0, b - a, 0, b]], dtype=np.int32)
        pkg.sdpa_rope_append_q8(q[a:b].to(dev), k[a:b].to(dev), v[a:b].to(dev), stored, torch.from_numpy(seq).to(dev), tabled)
        _, kb, wrote, _ = S.rope_append(q[a:b], k[a:b], v[a:b], rows, 1, seq, 0, table, (D // 2,))
        live, _, _, _ = S.step_rows(seq, b - a, rows, 1, 0)
        parts = [*S.q8_append(parts[0], parts[1], kb, wrote, seq, live, rows),
                 *S.q8_append(parts[2], parts[3], v[a:b], wrote, seq, live, rows)]
    for name, a, b in zip(pkg.Q8Store._fields, stored, parts):
        assert torch.equal(a.cpu(), torch.from_numpy(b)), name
    store = pkg.Q8Store(*(torch.from_numpy(t) for t in parts))
    seq = [[0, n, 0, n]]
    got, st = run_q8(q, store, seq, dev, causal=True)
    assert st == 0
    B.hold(got, q, store, seq, True)

    ks, vs = B.stores(store)
    whole = [np.zeros((rows, 1, Hkv, D)) for _ in range(2)]
    whole[0][:n, 0], whole[1][:n, 0] = S.f64(k), S.f64(v)
    ref, off, _ = B.bound(q, store, seq, True)
    exact, _, _ = O.sdpa_varlen(q, *whole, seq, True, 0, D ** -0.5, None, None)
    moved, _, _ = O.sdpa_varlen(q, ks, np.abs(vs - whole[1]), seq, True, 0, D ** -0.5, None, None)
    mag, _, _ = O.sdpa_varlen(q, ks, np.abs(whole[1]), seq, True, 0, D ** -0.5, None, None)
    ds = np.einsum("thgd,jhd->thgj", S.f64(q).reshape(n, Hkv, -1, D), (ks - whole[0])[:n, 0]) * D ** -0.5
    ds = np.abs(np.where(np.tri(n, dtype=bool)[:, None, None], ds, 0.0)).max(-1).reshape(n, Hq)[..., None]
    assert ds.max() < 0.2
    # |sum w' v' - sum w v| <= sum w' |v' - v| + sum |w' - w| |v|, and w is w' to a factor of exp(2 ds)
    far = off + moved + np.expm1(2 * ds) * mag
    assert (np.abs(S.f64(got) - exact) <= far).all()
