"""The shared-prefix calls as programs make them, beside test_gpu_shared.py: streams, workspaces,
scores that are not numbers, long stretches of tiles."""
import pytest
import torch

import relu_sparse_kv_gb300 as E
from test_gpu_shared import D, histogram, make, run

pytestmark = pytest.mark.gpu


def buffers_like(results):
    return [torch.full_like(t, -3) for t in results]


@pytest.mark.parametrize("B,Hkv,G,P,n", [(7, 4, 4, 3000, 50), (3, 2, 8, 129, 0)])
def test_a_stream_without_a_workspace(B, Hkv, G, P, n):
    """stream= with the workspace left to the call: the bits of the call on the current stream."""
    x = make(B, Hkv, G, P, n, 300 + B)
    alone = run(*x, P, n)
    side = torch.cuda.Stream()
    o = buffers_like(alone)
    side.wait_stream(torch.cuda.current_stream())
    E.embla_full_decode_shared(E.Shape(B, Hkv * G, Hkv, D, n, max(n, x[3].shape[2])), P, *x, *o, stream=side)
    torch.cuda.synchronize()
    assert E.embla_device_check() == 0
    assert all(torch.equal(a, b) for a, b in zip(alone, o))


def test_workspaces_of_calls_on_different_streams_do_not_meet():
    """Calls that make their own workspaces, alternately on the current stream and on one that waits
    only for the inputs: each workspace comes from its own stream's memory, so no call takes the
    records of one that still runs."""
    B, Hkv, G, P, n = 12, 4, 4, 6000, 40
    x = make(B, Hkv, G, P, n, 311)
    shape = E.Shape(B, Hkv * G, Hkv, D, n, n)
    alone = run(*x, P, n)
    outs = [buffers_like(alone) for _ in range(24)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for k, o in enumerate(outs):
        E.embla_full_decode_shared(shape, P, *x, *o, stream=side if k % 2 else None)
    torch.cuda.synchronize()
    assert E.embla_device_check() == 0
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(alone, o))


@pytest.mark.parametrize("G,Hkv,sstride", [(4, 4, 2304), (4, 2, 2301), (8, 2, 2304)])
def test_keys_without_a_number_rank_last(G, Hkv, sstride):
    """NaN key rows in the prefix and in own caches, all-zero rows with eps = 0, a NaN query head:
    scores, counts, histogram and selection are those of embla_full_decode on the whole contexts
    (scores to the tests' 60u of 128, which is 5e-4; the selection of the call's own scores exactly)."""
    B, P, n = 3, 2200, 100
    q, kp, vp, ko, vo = make(B, Hkv, G, P, n, 400 + G)
    kp[0, 5, 3] = float("nan")
    kp[1, 40:60] = 0.0
    kp[:, 700:1200] = float("nan")
    ko[1, 1, 99] = float("nan")
    ko[2, 0, :64] = 0.0
    q[0, 2] = float("nan")             # one head of a group: the others rank the keys
    q[2, Hkv * G - G:] = 0.0           # a whole group of zero queries: no score at all
    N = P + n
    out, ns, scores, hist = run(q, kp, vp, ko, vo, P, n, sstride, eps=0.0)
    K = torch.cat([kp[None].expand(B, -1, -1, -1), ko], 2).contiguous()
    V = torch.cat([vp[None].expand(B, -1, -1, -1), vo], 2).contiguous()
    out2, ns2, sig2 = torch.empty_like(out), torch.empty_like(ns), torch.empty(B, Hkv, N, device="cuda")
    E.embla_full_decode(E.Shape(B, Hkv * G, Hkv, D, N, N), q, K, V, out2, ns2, sig2, torch.empty_like(hist), eps=0.0)
    torch.cuda.synchronize()
    got = scores[..., :N]
    gone = got == -float("inf")
    assert torch.equal(gone, sig2 == -float("inf")) and torch.isfinite(got[~gone]).all()
    assert gone[:, 0, 5].all() and gone[:, 1, 40:60].all() and gone[1, 1, P + 99] and gone[2, 0, P:P + 64].all()
    assert gone[2, Hkv - 1].all() and not gone[0, 0].all()
    assert ((got - sig2)[~gone].abs() <= 5e-4).all()
    assert torch.equal(ns, (got > 0).sum(-1).int()) and torch.equal(hist, histogram(got))
    idx = torch.full((B, Hkv, 1152), -9, dtype=torch.int32, device="cuda")
    cnt = torch.empty(B, Hkv, dtype=torch.int32, device="cuda")
    E.embla_select_topk(E.Shape(B, Hkv * G, Hkv, D, N, sstride), scores, hist, idx, cnt)
    # equal scores: the smaller index first
    best = got[..., :N - 128].sort(dim=-1, descending=True, stable=True).indices[..., :1024].sort(-1).values
    want = torch.cat([best, torch.arange(N - 128, N, device="cuda").expand(B, Hkv, -1)], -1)
    numbers = ~gone[..., :N - 128].all(-1)  # (a unit without any number has no best keys)
    assert (cnt == 1152)[numbers].all() and torch.equal(idx.long()[numbers], want[numbers])
    assert E.embla_device_check() == 0


@pytest.mark.parametrize("Hkv,G,P,n,scores", [
    (1, 8, 262144, 0, True), (1, 4, 262144, 0, False),  # 2,048 prefix tiles per CTA
    (2, 8, 1000, 1500, True), (2, 4, 130, 900, False),  # own tiles of many sequences, two lists
])
def test_sums_of_many_tiles_do_not_drift(Hkv, G, P, n, scores):
    """A row block per SM, so that a CTA adds up all tiles of its sequences; values of one sign, so
    that errors add up too.  Bounds of the test file beside this one, with the sums as the kernel
    takes them: in tensor memory at most 64 tiles of 16 additions (8 steps, hi and lo) of at most
    4u each, the denominators 8 additions per tile and chain of at most u, and at most 64 fp32
    additions of such sums, whatever the length of the context."""
    B, u = 128 // G * E.embla_device_sm_count(), 2.0 ** -24
    g = torch.Generator(device="cuda").manual_seed(P + n)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()
    q, kp, vp = rnd(B, Hkv * G, D), rnd(Hkv, P, D), rnd(Hkv, P, D).abs()
    ko, vo = rnd(B, Hkv, n, D), rnd(B, Hkv, n, D).abs()
    out, ns, _, _ = run(q, kp, vp, ko, vo, P, n, sel=scores)
    norm = lambda x: x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    for b in (0, 1, 128 // G - 1, B // 2 + 3, B - 1):
        for h in range(Hkv):
            rows = slice(h * G, (h + 1) * G)
            k = norm(torch.cat([kp[h], ko[b, h]]).double())
            v = torch.cat([vp[h], vo[b, h]]).double()
            qq = norm(q[b, rows].double())
            s = (qq @ k.T).clamp(min=0)
            ds = 60 * u * (qq.abs() @ k.abs().T)
            w, dw = s.square(), 2 * s * ds + ds.square() + s.square() * (2.0 ** -17 + 2 * u)
            z = 1 + w.sum(-1, keepdim=True)
            num, want = w @ v, (w @ v) / z
            dnum = dw @ v + (4 * u * 16 * 64 + 64 * u) * num
            dz = dw.sum(-1, keepdim=True) + (8 * 64 + 64) * u * w.sum(-1, keepdim=True) + 4 * u * z
            tol = (dnum + want * dz) / z + 4 * u * want
            err = (out[b, rows].double() - want).abs()
            assert (err <= tol).all(), (b, h, float((err / want).max()), float((err / tol).max()))
            sure = (qq @ k.T).amax(0)
            assert int((sure > ds.amax(0)).sum()) <= int(ns[b, h]) <= int((sure > -ds.amax(0)).sum())


def test_sides_without_keys_may_be_none():
    """None for the prefix, or the own caches, of a call without keys there: the bits of the call with
    empty tensors."""
    for P, n in ((0, 300), (300, 0)):
        q, kp, vp, ko, vo = make(3, 2, 8, P, n, 51)
        planes = [t if t.numel() else None for t in (kp, vp, ko, vo)]
        sh, full = E.Shape(3, 16, 2, D, n, n), run(q, kp, vp, ko, vo, P, n)
        o = buffers_like(full)
        E.embla_full_decode_shared(sh, P, q, *planes, *o)
        idx = torch.arange(P + n, device="cuda", dtype=torch.int32).expand(3, 2, -1).contiguous()
        cnt = torch.full((3, 2), P + n, dtype=torch.int32, device="cuda")
        a, b = torch.empty_like(full[0]), torch.empty_like(full[0])
        E.embla_sparse_decode_shared(sh, P, q, kp, vp, ko, vo, idx, cnt, a)
        E.embla_sparse_decode_shared(sh, P, q, *planes, idx, cnt, b)
        torch.cuda.synchronize()
        assert E.embla_device_check() == 0
        assert all(torch.equal(s, t) for s, t in zip(full, o)) and torch.equal(a, b)


def test_sparse_weights_enter_the_value_sum_whole():
    """Two selected rows, scores 0 and s = -x y exactly (one nonzero element each), values powers of two:
    out = v p / (1 + p), p = 2^z, z = -tau2 x y.  With u = 2^-24: z carries 3u |z| (tau2 and the product),
    2.1u of p; exp2f 2 ulp, 4u; the value sum three additions (the parts of p) of 2u each at most, the
    sum of weights u and 6.1u p / (1 + p) of p, the division 2u: 18u of out in all, and 2u for the
    merges.  p in two bf16 parts alone would be off by up to 2^-18 = 64u."""
    B, Hkv, G, P, n, tau, u = 64, 4, 4, 3, 1, 0.5, 2.0 ** -24
    g = torch.Generator(device="cuda").manual_seed(8)
    q = torch.zeros(B, Hkv * G, D, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = (1 + torch.rand(B, Hkv * G, device="cuda", generator=g)).bfloat16()
    kp = torch.zeros(Hkv, P, D, device="cuda", dtype=torch.bfloat16)
    ko = torch.zeros(B, Hkv, n, D, device="cuda", dtype=torch.bfloat16)
    ko[..., 0] = -(torch.rand(B, Hkv, n, device="cuda", generator=g) * 0.5 + 0.1).bfloat16()
    two = lambda *s: (2.0 ** torch.randint(-3, 4, s, device="cuda", generator=g)).bfloat16()
    vp, vo = torch.zeros_like(kp), two(B, Hkv, n, D)
    idx = torch.tensor([1, P], dtype=torch.int32, device="cuda").expand(B, Hkv, 2).contiguous()
    cnt = torch.full((B, Hkv), 2, dtype=torch.int32, device="cuda")
    out = torch.empty(B, Hkv * G, D, device="cuda")
    E.embla_sparse_decode_shared(E.Shape(B, Hkv * G, Hkv, D, n, n), P, q, kp, vp, ko, vo, idx, cnt, out, tau=tau)
    torch.cuda.synchronize()
    s = q.view(B, Hkv, G, D)[..., 0].double() * ko[..., 0].double()
    p = torch.exp(tau * s)
    want = (p / (1 + p))[..., None] * vo[:, :, 0, None].double()
    err = ((out.view(B, Hkv, G, D).double() - want) / want).abs().max()
    assert err <= 20 * u, float(err / u)
