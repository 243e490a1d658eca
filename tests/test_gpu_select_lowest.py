"""The selection where fewer keys than it takes have a score above minus infinity (keys whose scores
were NaN for every head): the others come last, the smaller index first."""
import numpy as np
import pytest
import torch

import oracle
import relu_sparse_kv_gb300 as E
from helpers import order_key_np
from test_gpu_shared import D, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1500, 20000, 100000, 524289])  # one CTA, clusters, the streaming kernel
def test_keys_at_minus_infinity_fill_the_selection(n):
    rng = np.random.default_rng(n)
    B, Hkv = 2, 4
    sig = np.full((B, Hkv, n), -np.inf, dtype=np.float32)
    for u, some in enumerate((0, 1, 31, 1000, 1023, 1024, 1025, n)):  # numbers among the keys
        where = rng.permutation(n)[:some]
        sig[u // Hkv, u % Hkv, where] = rng.standard_normal(some)
    sig[0, 1, n - 5:] = 3.0
    sig[1, 0, 7] = -np.finfo(np.float32).max
    sig[1, 0, 8] = np.inf
    hist = np.stack([[np.bincount(order_key_np(sig[b, g]) >> 21, minlength=E.HIST_BINS)
                      for g in range(Hkv)] for b in range(B)]).astype(np.int32)
    idx = torch.full((B, Hkv, 1152), -1, dtype=torch.int32, device="cuda")
    cnt = torch.empty(B, Hkv, dtype=torch.int32, device="cuda")
    E.embla_select_topk(E.Shape(B, 16, Hkv, D, n, n), torch.from_numpy(sig).cuda(), torch.from_numpy(hist).cuda(),
                        idx, cnt)
    torch.cuda.synchronize()
    assert E.embla_device_check() == 0
    want, count = oracle.select_topk_batch(sig, n)
    assert np.array_equal(cnt.cpu().numpy(), count) and np.array_equal(idx.cpu().numpy(), want)


def test_nan_keys_fill_the_selection_behind_a_prefix():
    """More NaN keys than the selection leaves out: 1,152 keys all the same, the NaN ones last."""
    B, Hkv, G, P, n = 2, 4, 4, 2200, 100
    q, kp, vp, ko, vo = make(B, Hkv, G, P, n, 17)
    kp[:, 500:2000] = float("nan")
    q[1, :G] = float("nan")
    N = P + n
    _, _, scores, hist = run(q, kp, vp, ko, vo, P, n)
    idx = torch.full((B, Hkv, 1152), -9, dtype=torch.int32, device="cuda")
    cnt = torch.empty(B, Hkv, dtype=torch.int32, device="cuda")
    E.embla_select_topk(E.Shape(B, Hkv * G, Hkv, D, N, N), scores, hist, idx, cnt)
    torch.cuda.synchronize()
    want, count = oracle.select_topk_batch(scores.cpu().numpy(), N)
    assert np.array_equal(cnt.cpu().numpy(), count) and np.array_equal(idx.cpu().numpy(), want)
    assert (cnt == 1152).all() and E.embla_device_check() == 0


def test_nan_keys_rank_last_for_every_query_head():
    """Scores per query head with NaN key rows, zero key rows (eps = 0) and a NaN query head: minus
    infinity there, and the
    selection as the oracle makes it of those scores."""
    B, Hq, Hkv, n = 2, 16, 4, 2600
    g = torch.Generator(device="cuda").manual_seed(33)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()
    q, K, V = rnd(B, Hq, D), rnd(B, Hkv, n, D), rnd(B, Hkv, n, D)
    K[:, :, 11, 5] = float("nan")
    K[:, 1, 100:140] = 0.0
    K[:, 2, 300:2100] = float("nan")
    q[0, 1] = float("nan")
    before = K.clone()
    shape = E.Shape(B, Hq, Hkv, D, n, n)
    out, ns = torch.empty(B, Hq, D, device="cuda"), torch.empty(B, Hkv, dtype=torch.int32, device="cuda")
    hs = torch.empty(B, Hq, n, device="cuda")
    hh = torch.empty(B, Hq, E.HIST_BINS, dtype=torch.int32, device="cuda")
    E.embla_full_decode_head_scores(shape, q, K, V, out, ns, hs, hh, eps=0.0)
    idx = torch.full((B, Hq, 1152), -1, dtype=torch.int32, device="cuda")
    cnt = torch.empty(B, Hq, dtype=torch.int32, device="cuda")
    E.embla_select_topk_per_head(shape, hs, hh, idx, cnt)
    torch.cuda.synchronize()
    assert E.embla_device_check() == 0 and torch.equal(K.view(torch.int16), before.view(torch.int16))
    s = hs.cpu().numpy()
    gone = np.isneginf(s)
    assert not np.isnan(s).any() and gone[:, :, 11].all() and gone[:, 4:8, 100:140].all()
    assert gone[:, 8:12, 300:2100].all() and gone[0, 1].all() and gone[1, 1].sum() == 1
    assert np.array_equal(hh.cpu().numpy(), np.stack([[np.bincount(order_key_np(s[b, h]) >> 21, minlength=E.HIST_BINS)
                                                       for h in range(Hq)] for b in range(B)]))
    want, count = oracle.select_topk_batch(s, n)
    assert np.array_equal(cnt.cpu().numpy(), count) and np.array_equal(idx.cpu().numpy(), want)
