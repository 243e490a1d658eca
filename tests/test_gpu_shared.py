"""Decode behind a shared prefix (embla_full_decode_shared, embla_sparse_decode_shared) against the
definitions in 64 bits, sequence by sequence on prefix and own keys put together.

Tolerances, from the arithmetic of the kernels (u = 2^-24, half a step of fp32):
  scores   s' = dot rk rq: the dot product is 8 tensor-core steps of 16 exact bf16 products, each
           step summed and added with at most 4u of the magnitudes A = sum |q^ k^| (alignment of
           the 17 terms), so 32u A; the two norms carry 2^-22 each from rsqrtf and 8u from their
           sums of squares, the products 2u: ds = (32u + 2 * (4u + 8u) + 4u) A = 60u A.
  weights  dw = 2 s ds + ds^2, plus 2^-17 w for the hi + lo split (each bf16 rounding is 2^-9 of
           what is left) and 2u w.
  sums     per 16-key step 2 (hi and lo) additions of at most 4u of the running magnitude, and
           one per record: with n_add of them the sum is off by at most 4u n_add sum w |v|; the
           denominators the same over n_add / 2.
  out      the sum's error over the normaliser, plus |out| times the normaliser's relative error."""
import numpy as np
import pytest
import torch

import gen
import oracle
import relu_sparse_kv_gb300 as E
from helpers import assert_close, to_dev

pytestmark = pytest.mark.gpu
D = 128
U = 2.0 ** -24
EPS = 1e-6


def make(B, Hkv, G, P, n, seed, pstride=None, ncap=None, shift=1.2):
    """Queries that share a direction per KV head and keys that turn away from it (a small part of
    the scores is positive); rows past P and n are NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)
    pstride, ncap = pstride or P, ncap or n
    u = torch.nn.functional.normalize(r(Hkv, D), dim=-1)
    q = (r(B, Hkv, G, D) + 8.0 * u[None, :, None]).bfloat16().view(B, Hkv * G, D)
    nan = float("nan")
    kp, vp = (torch.full((Hkv, pstride, D), nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ko, vo = (torch.full((B, Hkv, ncap, D), nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kp[:, :P] = (r(Hkv, P, D) - shift * u[:, None]).bfloat16()
    vp[:, :P] = r(Hkv, P, D).bfloat16()
    ko[:, :, :n] = (r(B, Hkv, n, D) - shift * u[None, :, None]).bfloat16()
    vo[:, :, :n] = r(B, Hkv, n, D).bfloat16()
    return q, kp, vp, ko, vo


def reference(q, kp, vp, ko, vo, P, n, alpha, c, eps):
    """(out, out's tolerance, scores of every key, their tolerance) in 64 bits."""
    B, Hq, _ = q.shape
    Hkv = kp.shape[0]
    G = Hq // Hkv
    norm = lambda x: x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    sig = torch.zeros(B, Hkv, P + n, dtype=torch.float64, device="cuda")
    stol = torch.zeros_like(sig)
    for b in range(B):
        for g in range(Hkv):
            k = norm(torch.cat([kp[g, :P], ko[b, g, :n]]).double())
            v = torch.cat([vp[g, :P], vo[b, g, :n]]).double()
            qq = norm(q[b, g * G:(g + 1) * G].double())
            s = qq @ k.T
            ds = 60 * U * (qq.abs() @ k.abs().T)
            w = s.clamp(min=0).square().nan_to_num(nan=0.0)
            dw = (2 * s.clamp(min=0) * ds + ds.square()).nan_to_num(nan=0.0) + w * (2.0 ** -17 + 2 * U)
            # a key of weight zero contributes nothing, whatever its value row holds; a weight that
            # may be zero or not (|s| within ds of it) moves the sum by dw |v| at most
            dead = (w == 0).all(0)
            v = torch.where(dead[:, None], 0.0, v)
            av = torch.where(torch.isfinite(v), v.abs(), 0.0)
            z = c / alpha ** 2 + w.sum(-1, keepdim=True)
            n_add = 2 * ((P + 127) // 128 + (n + 127) // 128) * 8 + 160
            live = z > 0
            # 0 * (inf or NaN) is not formed: keys other heads need are cut per head
            num = torch.stack([torch.where(w[i][:, None] > 0, w[i][:, None] * v, 0.0).sum(0) for i in range(G)])
            mag = w @ av
            dnum = dw @ av + 4 * U * n_add * mag
            dz = dw.sum(-1, keepdim=True) + 2 * U * n_add * w.sum(-1, keepdim=True) + 4 * U * z
            h = slice(g * G, (g + 1) * G)
            o = torch.where(live, num / z, 0.0)
            out[b, h] = o
            tol[b, h] = torch.where(live, (dnum + o.abs() * dz) / z, 0.0) + 4 * U * o.abs()
            sig[b, g] = alpha * s.nan_to_num(nan=-float("inf")).amax(0)
            stol[b, g] = alpha * ds.amax(0) + 2 * U * sig[b, g].abs()
    return out, tol, sig, stol


def run(q, kp, vp, ko, vo, P, n, sstride=None, sel=True, alpha=1.0, c=1.0, eps=EPS, workspace=None):
    B, Hq, _ = q.shape
    Hkv = kp.shape[0]
    shape = E.Shape(B, Hq, Hkv, D, n, ko.shape[2])
    out = torch.full((B, Hq, D), float("nan"), device="cuda")
    ns = torch.full((B, Hkv), -1, dtype=torch.int32, device="cuda")
    scores = torch.full((B, Hkv, sstride or P + n), 777.0, device="cuda") if sel else None
    hist = torch.full((B, Hkv, E.HIST_BINS), -1, dtype=torch.int32, device="cuda") if sel else None
    E.embla_full_decode_shared(shape, P, q, kp, vp, ko, vo, out, ns, scores, hist, alpha=alpha, c=c, eps=eps,
                               workspace=workspace)
    torch.cuda.synchronize()
    assert E.embla_device_check() == 0
    return out, ns, scores, hist


def histogram(scores):
    """The 2048-bin histogram of order keys that embla_select_topk reads."""
    s = torch.where(scores == 0, torch.zeros_like(scores), scores)
    bits = s.contiguous().view(torch.int32).long()
    key = torch.where(bits < 0, -1 - bits, bits + (1 << 31)) >> 21
    h = torch.zeros(*scores.shape[:2], E.HIST_BINS, dtype=torch.int64, device="cuda")
    return h.scatter_add_(2, key, torch.ones_like(key)).int()


def check(inputs, P, n, sstride=None, alpha=1.0, c=1.0, eps=EPS):
    out, ns, scores, hist = run(*inputs, P, n, sstride, True, alpha, c, eps)
    want, tol, sig, stol = reference(*inputs, P, n, alpha, c, eps)
    bad = ~((out.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((out.double() - want).abs() / tol.clamp(min=1e-30)).max()))
    got = scores[..., :P + n]
    assert ((got.double() - sig).abs() <= stol).all()
    assert (scores[..., P + n:] == 777.0).all()
    # counts and bins are those of the scores the call returned
    assert torch.equal(ns, (got > 0).sum(-1).int())
    assert torch.equal(hist, histogram(got))
    return out, ns, scores, hist


CASES = [
    # B, Hkv, G, P, n, prefix stride, cache stride, score stride
    (1, 1, 4, 1, 0, 1, 1, 1),
    (1, 4, 4, 0, 1, 1, 1, 4),
    (2, 2, 8, 127, 1, 130, 2, 128),
    (3, 4, 4, 128, 128, 128, 128, 256),
    (4, 4, 4, 129, 17, 200, 40, 149),       # odd strides: scores stored one by one
    (5, 2, 8, 1000, 130, 1000, 131, 1136),
    (16, 2, 8, 640, 0, 640, 1, 640),        # one full row block of groups of 8, no own keys
    (17, 2, 8, 513, 33, 520, 64, 552),      # a second row block of one sequence
    (33, 4, 4, 2048, 300, 2048, 300, 2352),
    (40, 1, 4, 0, 257, 1, 300, 264),        # no prefix: own keys only
    (70, 4, 4, 384, 5, 384, 8, 392),        # three row blocks, the last of six
    (2, 4, 4, 20000, 700, 20000, 1000, 20704),  # pieces of many tiles
    (4, 4, 4, 1024, 3001, 1024, 3001, 4032),    # own contexts longer than the prefix
    (2500, 1, 8, 129, 2, 130, 3, 132),          # more row blocks than SMs
]


@pytest.mark.parametrize("B,Hkv,G,P,n,pstride,ncap,sstride", CASES)
def test_full_shared_matches_the_definition(B, Hkv, G, P, n, pstride, ncap, sstride):
    check(make(B, Hkv, G, P, n, B + P + n, pstride, ncap), P, n, sstride)


@pytest.mark.parametrize("alpha,c,eps", [(0.7, 0.0, 1e-6), (3.0, 0.5, 1e-2), (1e-3, 1.0, 1e-6)])
def test_full_shared_scalars(alpha, c, eps):
    check(make(6, 2, 8, 700, 50, 11), 700, 50, None, alpha, c, eps)


def test_full_shared_without_selection_outputs_and_with_a_used_workspace():
    """Bits do not depend on the selection outputs being asked for or on what a workspace held."""
    x = make(9, 4, 4, 3000, 90, 21)
    a = run(*x, 3000, 90, 3096)
    shape = E.Shape(9, 16, 4, D, 90, 90)
    need = E.embla_full_decode_shared_workspace_size(shape, 3000)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN records
    for sel in (True, False, True):
        b = run(*x, 3000, 90, 3096, sel, workspace=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        if sel:
            assert torch.equal(a[2], b[2]) and torch.equal(a[3], b[3])
    with pytest.raises(E.EmblaError) as err:
        run(*x, 3000, 90, 3096, workspace=ws[:need - 16])
    assert err.value.status == 3


def test_full_shared_with_buffers_on_sixteen_bytes_only():
    """Every buffer 16 bytes off a 32-byte boundary: the same bits as with wider alignment."""
    B, Hkv, G, P, n = 5, 4, 4, 700, 45
    x = make(B, Hkv, G, P, n, 23)
    a = run(*x, P, n, 752)

    def shifted(t, fill=None):
        raw = torch.empty(t.numel() * t.element_size() + 32, dtype=torch.uint8, device="cuda")
        start = (16 - raw.data_ptr()) % 32
        v = raw[start:start + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        assert v.data_ptr() % 32 == 16
        return v.copy_(t) if fill is None else v.fill_(fill)

    shape = E.Shape(B, Hkv * G, Hkv, D, n, n)
    o = [shifted(t, 777) for t in a]
    ws = shifted(torch.empty(E.embla_full_decode_shared_workspace_size(shape, P), dtype=torch.uint8, device="cuda"))
    E.embla_full_decode_shared(shape, P, *[shifted(t) for t in x], *o, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(a, o))


def test_planes_past_32_bit_offsets():
    """Prefix and own planes more than 2^31 elements apart (and rows of the own caches past 2^32
    bytes): the definition on the rows that are there, for both calls."""
    B, Hkv, G, P, n, stride = 2, 2, 8, 300, 40, (1 << 24) + 5
    q, kp, vp, ko, vo = make(B, Hkv, G, P, n, 27)
    far = []
    for t, planes in ((kp, (Hkv,)), (vp, (Hkv,)), (ko, (B, Hkv)), (vo, (B, Hkv))):
        big = torch.empty(*planes, stride, D, dtype=torch.bfloat16, device="cuda")
        big[..., :t.shape[-2], :] = t
        big[..., t.shape[-2]:t.shape[-2] + 200, :] = float("nan")
        far.append(big)
    assert far[2][1, 1].data_ptr() - far[2].data_ptr() > 1 << 33
    check((q, *far), P, n, 344)
    g = torch.Generator(device="cuda").manual_seed(2)
    idx = torch.randint(0, P + n, (B, Hkv, 64), device="cuda", generator=g, dtype=torch.int32)
    cnt = torch.full((B, Hkv), 64, dtype=torch.int32, device="cuda")
    out = torch.empty(B, Hkv * G, D, device="cuda")
    E.embla_sparse_decode_shared(E.Shape(B, Hkv * G, Hkv, D, n, stride), P, q, *far, idx, cnt, out)
    ref, tol = sparse_reference(q, kp, vp, ko, vo, P, idx, cnt, D ** -0.5)
    assert ((out.double() - ref).abs() <= tol).all()


def test_full_shared_agrees_with_the_decode_of_whole_contexts():
    """The same contexts as B separate caches through embla_full_decode: scores agree to fp32
    rounding (60u of sum |q^ k^| <= 128 on either side), outputs to both calls' bounds."""
    B, Hkv, G, P, n = 5, 4, 4, 1500, 77
    x = make(B, Hkv, G, P, n, 31)
    out, ns, scores, _ = run(*x, P, n)
    q, kp, vp, ko, vo = x
    K = torch.cat([kp[None].expand(B, -1, -1, -1), ko], 2).contiguous()
    V = torch.cat([vp[None].expand(B, -1, -1, -1), vo], 2).contiguous()
    out2, ns2 = torch.empty_like(out), torch.empty_like(ns)
    sel2 = torch.empty(B, Hkv, P + n, device="cuda")
    h2 = torch.empty(B, Hkv, E.HIST_BINS, dtype=torch.int32, device="cuda")
    E.embla_full_decode(E.Shape(B, Hkv * G, Hkv, D, P + n, P + n), q, K, V, out2, ns2, sel2, h2)
    torch.cuda.synchronize()
    _, tol, _, stol = reference(*x, P, n, 1.0, 1.0, EPS)
    assert ((scores - sel2).double().abs() <= 2 * stol).all()
    assert ((out - out2).double().abs() <= 2 * tol + 1e-30).all()
    assert int((ns - ns2).abs().max()) <= int((scores.abs() <= 2 * stol).sum())


def test_no_survivor_and_no_keys():
    """Keys opposite to every query: nothing weighs, with c = 0 the outputs are 0.  No keys at all:
    zero outputs, counts and histogram."""
    q, kp, vp, ko, vo = make(3, 2, 8, 300, 20, 41)
    u = torch.nn.functional.normalize(torch.randn(2, D, device="cuda"), dim=-1)
    q = (5 * u.repeat_interleave(8, 0)[None].expand(3, -1, -1)).bfloat16().contiguous()
    kp = (-2 * u[:, None].expand(2, 300, D)).bfloat16().contiguous()
    ko = (-3 * u[None, :, None].expand(3, 2, 20, D)).bfloat16().contiguous()
    out, ns, scores, hist = run(q, kp, vp, ko, vo, 300, 20, c=0.0)
    assert (out == 0).all() and (ns == 0).all() and (scores < 0).all()
    e = torch.empty(2, 0, D, dtype=torch.bfloat16, device="cuda")
    eo = torch.empty(3, 2, 0, D, dtype=torch.bfloat16, device="cuda")
    out, ns, scores, hist = run(q, e, e, eo, eo, 0, 0, sstride=8)
    assert (out == 0).all() and (ns == 0).all() and (hist == 0).all() and (scores == 777.0).all()


@pytest.mark.parametrize("G,Hkv", [(4, 4), (8, 2)])
def test_values_of_dead_keys_may_be_anything(G, Hkv):
    """Infinite and NaN value rows at keys that no head of a sequence weighs above zero leave that
    sequence's outputs as they are; a head that does weigh them gets the infinity or NaN."""
    B, P, n = 6, 900, 140
    x = make(B, Hkv, G, P, n, 51, shift=2.85)
    q, kp, vp, ko, vo = x
    _, _, sig, _ = reference(*x, P, n, 1.0, 1.0, EPS)
    plain = run(*x, P, n)[0]
    # a prefix key dead for every sequence of KV head 0, and an own key of sequence 2
    dead = int((sig[:, 0, :P] < -0.5).all(0).nonzero()[0])
    own = int((sig[2, 1, P:] < -0.5).nonzero()[0])
    vp[0, dead] = float("nan")
    vo[2, 1, own] = float("-inf")
    out = check(x, P, n)[0]
    assert torch.isfinite(out).all()
    # a key alive for one sequence at least: its heads see the NaN, all others do not
    alive = int((sig[3, 0, :P] > 0.5).nonzero()[0])
    vp[0, alive, 7] = float("nan")
    out = run(*x, P, n)[0]
    want, _, _, _ = reference(*x, P, n, 1.0, 1.0, EPS)
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.isnan(out).any()
    rest = ~torch.isnan(out)
    assert ((out - plain)[rest].abs() <= 1e-4 * plain[rest].abs() + 1e-5).all()
    # two values of opposite infinite sign of one head: NaN; of the same sign: infinite
    vp[0, alive, 7] = float("inf")
    out = run(*x, P, n)[0]
    want, _, _, _ = reference(*x, P, n, 1.0, 1.0, EPS)
    assert torch.equal(torch.isinf(out), torch.isinf(want)) and not torch.isnan(out).any()


def test_nan_keys_and_queries_stay_their_own():
    """A NaN key weighs nothing; a NaN query row of one head leaves the other heads alone."""
    B, Hkv, G, P, n = 3, 2, 8, 300, 30
    q, kp, vp, ko, vo = make(B, Hkv, G, P, n, 61)
    base = run(q, kp, vp, ko, vo, P, n)
    q2, ko2 = q.clone(), ko.clone()
    q2[1, 3] = float("nan")
    ko2[2, 0, 5] = float("nan")
    out, ns, _, _ = run(q2, kp, vp, ko2, vo, P, n)
    same = torch.ones(B, Hkv * G, dtype=torch.bool, device="cuda")
    same[1, 3] = False
    same[2, :G] = False
    assert torch.equal(out[same], base[0][same])
    assert (out[1, 3] == 0).all()  # no weight, c = 1
    k3 = torch.cat([ko[2, 0, :5], ko[2, 0, 6:]])[None, None]
    ref, tol, _, _ = reference(q[2:3, :G], kp[:1], vp[:1], k3, torch.cat([vo[2, 0, :5], vo[2, 0, 6:]])[None, None],
                               P, n - 1, 1.0, 1.0, EPS)
    assert ((out[2, :G].double() - ref[0]).abs() <= tol[0]).all()


@pytest.mark.parametrize("Hq,P", [(16, 1500), (16, 2048 - 128), (32, 1), (32, 2047)])
def test_one_sequence_split_anywhere_matches_the_oracle(Hq, P):
    """A generated context (scores and selection kept away from ties) cut into a prefix and own keys:
    the oracle's survivor counts and selection exactly, its outputs to the usual tolerance."""
    n_all, Hkv = 2048, 4
    fl = gen.make_full_layer(seed=7, layer=0, B=1, Hq=Hq, Hkv=Hkv, D=D, n=n_all, pattern="bernoulli",
                             frac=0.3, sparse_layers=(1,))
    q, K, V = to_dev(fl.q), to_dev(fl.K), to_dev(fl.V)
    kp, vp = K[0, :, :P].contiguous(), V[0, :, :P].contiguous()
    ko, vo = K[:, :, P:].contiguous(), V[:, :, P:].contiguous()
    n = n_all - P
    out, ns, scores, hist = run(q, kp, vp, ko, vo, P, n)
    ref_out, ref_sig, ref_ns = oracle.full_decode_batch(fl.q, fl.K, fl.V, n_all)
    assert_close(out.cpu().numpy(), ref_out, what="shared full output")
    assert np.array_equal(ns.cpu().numpy(), ref_ns)
    idx = torch.empty(1, Hkv, 1152, dtype=torch.int32, device="cuda")
    cnt = torch.empty(1, Hkv, dtype=torch.int32, device="cuda")
    E.embla_select_topk(E.Shape(1, Hq, Hkv, D, n_all, n_all), scores, hist, idx, cnt)
    sout = torch.empty(1, Hq, D, device="cuda")
    qs = to_dev(fl.sparse_q[0])
    E.embla_sparse_decode_shared(E.Shape(1, Hq, Hkv, D, n, n), P, qs, kp, vp, ko, vo, idx, cnt, sout)
    torch.cuda.synchronize()
    ref_idx, ref_cnt = oracle.select_topk_batch(ref_sig, n_all)
    assert np.array_equal(cnt.cpu().numpy(), ref_cnt) and np.array_equal(idx.cpu().numpy(), ref_idx)
    assert_close(sout.cpu().numpy(), oracle.sparse_decode_batch(fl.sparse_q[0], fl.K, fl.V, ref_idx, ref_cnt),
                 what="shared sparse output")


def test_two_calls_on_two_streams_at_once():
    """Two batches behind different prefixes, each with its own workspace on its own stream, eight
    calls of each in flight together: the bits of the calls made alone."""
    sizes = [(12, 4, 4, 5000, 64), (9, 2, 8, 7000, 33)]
    xs = [make(B, Hkv, G, P, n, 200 + B) for B, Hkv, G, P, n in sizes]
    alone = [run(*x, P, n) for x, (_, _, _, P, n) in zip(xs, sizes)]
    streams = [torch.cuda.Stream() for _ in sizes]
    got = []
    for x, (B, Hkv, G, P, n) in zip(xs, sizes):
        shape = E.Shape(B, Hkv * G, Hkv, D, n, n)
        ws = torch.empty(E.embla_full_decode_shared_workspace_size(shape, P), dtype=torch.uint8, device="cuda")
        got.append((shape, ws, [torch.full_like(t, -3) for t in alone[len(got)]]))
    torch.cuda.synchronize()
    for _ in range(8):
        for x, (_, _, _, P, _), st, (shape, ws, o) in zip(xs, sizes, streams, got):
            E.embla_full_decode_shared(shape, P, *x, *o, workspace=ws, stream=st)
    torch.cuda.synchronize()
    assert E.embla_device_check() == 0
    for a, (_, _, o) in zip(alone, got):
        assert all(torch.equal(s, t) for s, t in zip(a, o))


def chain(x, P, n, sstride, topk=1024, recent=128):
    """full -> select -> sparse, as a block of layers runs behind a shared prefix."""
    q, kp, vp, ko, vo = x
    B, Hq, _ = q.shape
    Hkv = kp.shape[0]
    out, ns, scores, hist = run(*x, P, n, sstride)
    idx = torch.full((B, Hkv, topk + recent), -9, dtype=torch.int32, device="cuda")
    cnt = torch.empty(B, Hkv, dtype=torch.int32, device="cuda")
    E.embla_select_topk(E.Shape(B, Hq, Hkv, D, P + n, sstride), scores, hist, idx, cnt, topk, recent)
    sout = torch.full((B, Hq, D), float("nan"), device="cuda")
    E.embla_sparse_decode_shared(E.Shape(B, Hq, Hkv, D, n, ko.shape[2]), P, q, kp, vp, ko, vo, idx, cnt, sout)
    torch.cuda.synchronize()
    assert E.embla_device_check() == 0
    return scores, idx, cnt, sout


def sparse_reference(q, kp, vp, ko, vo, P, idx, cnt, tau):
    """Softmax over the selected rows in 64 bits, and its tolerance: z carries 40u of
    tau sum |q k| (8 steps of 4u, the scale and the base change) and exp2 2 ulp, so every
    probability e = dz + 8u; the split of P 2^-17; sums of at most 1152 terms in blocks 100u."""
    B, Hq, _ = q.shape
    Hkv = kp.shape[0]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    for b in range(B):
        for g in range(Hkv):
            j = idx[b, g, :int(cnt[b, g])].long()
            if j.numel() == 0:
                continue
            k = torch.cat([kp[g, :P], ko[b, g]])[j].double()
            v = torch.cat([vp[g, :P], vo[b, g]])[j].double()
            qq = q[b, g * G:(g + 1) * G].double()
            p = torch.softmax(tau * (qq @ k.T), -1)
            e = torch.expm1(2 * (40 * U * abs(tau) * (qq.abs() @ k.abs().T).amax(-1, keepdim=True) + 8 * U))
            h = slice(g * G, (g + 1) * G)
            out[b, h] = p @ v
            tol[b, h] = (e + 2.0 ** -17 + 100 * U) * (p @ v.abs())
    return out, tol


@pytest.mark.parametrize("B,Hkv,G,P,n,sstride", [
    (2, 4, 4, 3000, 100, 3104),    # recent keys reach into the prefix
    (3, 2, 8, 2500, 400, 2904),
    (2, 4, 4, 600, 40, 640),       # every key selected
    (20, 4, 4, 1500, 1, 1504),
])
def test_full_then_selection_then_sparse(B, Hkv, G, P, n, sstride):
    x = make(B, Hkv, G, P, n, 71 + P)
    scores, idx, cnt, sout = chain(x, P, n, sstride)
    N = P + n
    old = max(0, N - 128)
    top = min(1024, old)
    assert (cnt == top + N - old).all()
    best = scores[..., :old].double()
    # ties (none in random scores) aside, the top scores and the newest keys
    want = torch.cat([best.topk(top, -1).indices.sort(-1).values,
                      torch.arange(old, N, device="cuda").expand(B, Hkv, -1)], -1)
    assert torch.equal(idx[..., :top + N - old].long(), want)
    ref, tol = sparse_reference(*x, P, idx, cnt, D ** -0.5)
    assert ((sout.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("B,Hkv,G,P,n,stride,counts", [
    (1, 1, 4, 5, 0, 8, [3]), (3, 2, 8, 0, 50, 64, [0, 50, 1, 17, 16, 33]), (2, 4, 4, 77, 9, 1152, [86, 1, 0, 85, 64, 2, 9, 10]),
    (40, 4, 4, 1200, 30, 1152, None), (80, 4, 4, 300, 3, 300, None), (2, 2, 8, 3000, 100, 7001, [7001, 0, 6000, 1153]),
])
def test_sparse_shared_matches_the_definition(B, Hkv, G, P, n, stride, counts):
    """Any list of keys in any order, the same key twice, empty lists; entries past the count are
    not read as rows."""
    q, kp, vp, ko, vo = make(B, Hkv, G, P, n, 81 + B, P + 3, n + 2)
    g = torch.Generator(device="cuda").manual_seed(B)
    idx = torch.randint(0, P + n, (B, Hkv, stride), device="cuda", generator=g, dtype=torch.int32)
    cnt = torch.randint(0, stride + 1, (B, Hkv), device="cuda", generator=g, dtype=torch.int32)
    if counts:
        cnt = torch.tensor(counts, dtype=torch.int32, device="cuda").view(B, Hkv)
    past = torch.arange(stride, device="cuda") >= cnt[..., None]
    idx = torch.where(past, torch.full_like(idx, -5), idx)
    out = torch.full((B, Hkv * G, D), float("nan"), device="cuda")
    E.embla_sparse_decode_shared(E.Shape(B, Hkv * G, Hkv, D, n, n + 2), P, q, kp, vp, ko, vo, idx, cnt, out)
    torch.cuda.synchronize()
    assert E.embla_device_check() == 0
    ref, tol = sparse_reference(q, kp, vp, ko, vo, P, idx, cnt, D ** -0.5)
    assert ((out.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("P,n", [(0, 40), (40, 0), (0, 0)])
def test_sides_without_keys_need_no_memory(P, n):
    """Null planes for the side without keys: lists that end inside a block, empty ones, and (no keys
    at all) only empty ones; the full layer on the same contexts."""
    B, Hkv, G = 3, 2, 8
    q, kp, vp, ko, vo = make(B, Hkv, G, P, n, 101, P, n)
    g = torch.Generator(device="cuda").manual_seed(6)
    idx = torch.randint(0, max(1, P + n), (B, Hkv, 50), device="cuda", generator=g, dtype=torch.int32)
    cnt = torch.tensor([50, 1, 0, 17, 16, 33] if P + n else [0] * 6, dtype=torch.int32, device="cuda").view(B, Hkv)
    for t, keys in ((kp, P), (vp, P), (ko, n), (vo, n)):
        assert keys > 0 or t.data_ptr() == 0
    out = torch.full((B, Hkv * G, D), float("nan"), device="cuda")
    sh = E.Shape(B, Hkv * G, Hkv, D, n, n)
    E.embla_sparse_decode_shared(sh, P, q, kp, vp, ko, vo, idx, cnt, out)
    full, ns = torch.full_like(out, float("nan")), torch.full((B, Hkv), -1, dtype=torch.int32, device="cuda")
    E.embla_full_decode_shared(sh, P, q, kp, vp, ko, vo, full, ns)
    torch.cuda.synchronize()
    assert E.embla_device_check() == 0
    if P + n == 0:
        assert (out == 0).all() and (full == 0).all() and (ns == 0).all()
        return
    ref, tol = sparse_reference(q, kp, vp, ko, vo, P, idx, cnt, D ** -0.5)
    assert ((out.double() - ref).abs() <= tol).all()
    assert torch.isfinite(full).all() and (ns <= P + n).all() and (ns >= 0).all()


def test_sparse_shared_agrees_with_the_call_on_whole_caches():
    """embla_sparse_decode on the contexts put together: both are within their bounds of the
    definition (the shared call carries one more part of the probabilities)."""
    B, Hkv, G, P, n = 4, 4, 4, 1000, 200
    q, kp, vp, ko, vo = make(B, Hkv, G, P, n, 91)
    g = torch.Generator(device="cuda").manual_seed(4)
    idx = torch.rand(B, Hkv, P + n, device="cuda", generator=g).topk(1152).indices.sort().values.int()
    cnt = torch.full((B, Hkv), 1152, dtype=torch.int32, device="cuda")
    a = torch.empty(B, Hkv * G, D, device="cuda")
    b = torch.empty_like(a)
    E.embla_sparse_decode_shared(E.Shape(B, Hkv * G, Hkv, D, n, n), P, q, kp, vp, ko, vo, idx, cnt, a)
    K = torch.cat([kp[None].expand(B, -1, -1, -1), ko], 2).contiguous()
    V = torch.cat([vp[None].expand(B, -1, -1, -1), vo], 2).contiguous()
    E.embla_sparse_decode(E.Shape(B, Hkv * G, Hkv, D, P + n, P + n), q, K, V, idx, cnt, b)
    torch.cuda.synchronize()
    _, tol = sparse_reference(q, kp, vp, ko, vo, P, idx, cnt, D ** -0.5)
    assert ((a - b).double().abs() <= 2 * tol).all()


def test_sparse_shared_flags_indices_outside_the_context():
    B, Hkv, G, P, n = 2, 2, 8, 100, 10
    q, kp, vp, ko, vo = make(B, Hkv, G, P, n, 95)
    idx = torch.arange(32, device="cuda", dtype=torch.int32).expand(B, Hkv, 32).contiguous()
    idx[0, 0, 3], idx[1, 1, 31] = P + n, -1
    cnt = torch.full((B, Hkv), 32, dtype=torch.int32, device="cuda")
    out = torch.empty(B, Hkv * G, D, device="cuda")
    E.embla_sparse_decode_shared(E.Shape(B, Hkv * G, Hkv, D, n, n), P, q, kp, vp, ko, vo, idx, cnt, out)
    assert E.embla_device_check() == 1
    assert E.embla_device_check() == 0
    keep = idx.clone()
    keep[0, 0, 3:31] = idx[0, 0, 4:32]
    cnt[0, 0] = cnt[1, 1] = 31
    ref, tol = sparse_reference(q, kp, vp, ko, vo, P, keep, cnt, D ** -0.5)
    assert ((out.double() - ref).abs() <= tol).all()


def test_the_block_in_a_graph_on_a_side_stream():
    """full -> select -> sparse captured once and replayed on new queries and own keys: the same
    bits as the calls made one by one; two graphs take turns with one workspace."""
    B, Hkv, G, P, n = 6, 4, 4, 2500, 60
    x = make(B, Hkv, G, P, n, 101)
    q, kp, vp, ko, vo = x
    N = P + n
    shape, sel_shape = E.Shape(B, 16, Hkv, D, n, n), E.Shape(B, 16, Hkv, D, N, 2560)
    ws = torch.empty(E.embla_full_decode_shared_workspace_size(shape, P), dtype=torch.uint8, device="cuda")
    dev = dict(device="cuda")

    def buffers():
        return (torch.zeros(B, 16, D, **dev), torch.zeros(B, Hkv, dtype=torch.int32, **dev),
                torch.zeros(B, Hkv, 2560, **dev), torch.zeros(B, Hkv, E.HIST_BINS, dtype=torch.int32, **dev),
                torch.zeros(B, Hkv, 1152, dtype=torch.int32, **dev), torch.zeros(B, Hkv, dtype=torch.int32, **dev),
                torch.zeros(B, 16, D, **dev))

    def block(o):
        E.embla_full_decode_shared(shape, P, q, kp, vp, ko, vo, *o[:4], workspace=ws)
        E.embla_select_topk(sel_shape, o[2], o[3], o[4], o[5])
        E.embla_sparse_decode_shared(shape, P, q, kp, vp, ko, vo, o[4], o[5], o[6])

    plain, one, two = buffers(), buffers(), buffers()
    side = torch.cuda.Stream()
    graphs = []
    for o in (one, two):
        graph = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            block(o)
        graphs.append(graph)
    g = torch.Generator(device="cuda").manual_seed(6)
    for _ in range(3):
        q.copy_(torch.randn(B, 16, D, device="cuda", generator=g).bfloat16())
        ko.copy_(torch.randn(B, Hkv, n, D, device="cuda", generator=g).bfloat16())
        for graph in graphs:
            graph.replay()
        block(plain)
        torch.cuda.synchronize()
        for a, b, c in zip(plain, one, two):
            assert torch.equal(a, b) and torch.equal(a, c)
    assert E.embla_device_check() == 0


def test_prompt_through_the_8_bit_store_to_a_shared_prefix():
    """A prompt's rows quantised into the 8-bit caches, read back as the bf16 prefix of a batch, and
    decoded: the result is the definition on the rows that the codes stand for."""
    B, Hkv, G, P, n = 5, 2, 8, 1111, 20
    q, kp, vp, ko, vo = make(B, Hkv, G, P, n, 111)
    store = E.Shape(1, G * Hkv, Hkv, D, P, 1200)
    codes = [torch.zeros(1, Hkv, 1200, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(1, Hkv, 1200, device="cuda") for _ in range(2)]
    E.embla_quantize_kv_e4m3(store, 0, kp[None], vp[None], codes[0], scales[0], codes[1], scales[1])
    kb, vb = torch.full_like(kp, float("nan")), torch.full_like(vp, float("nan"))
    E.embla_dequantize_kv_e4m3(store, 0, codes[0], scales[0], codes[1], scales[1], kb[None], vb[None])
    check((q, kb, vb, ko, vo), P, n)
    stands = lambda c, s: (c[0, :, :P].view(torch.float8_e4m3fn).float() * s[0, :, :P, None]).bfloat16()
    assert torch.equal(kb, stands(codes[0], scales[0])) and torch.equal(vb, stands(codes[1], scales[1]))


def test_refusals_on_device_tensors():
    q, kp, vp, ko, vo = make(2, 2, 8, 100, 10, 121)
    with pytest.raises(ValueError):
        run(q, kp, vp, ko, vo, 101, 10)            # the prefix holds 100 rows
    with pytest.raises(E.EmblaError) as err:
        run(q, kp, vp, ko, vo, 100, 11, 120)       # the own caches hold 10
    assert err.value.status == 1
    with pytest.raises(E.EmblaError):
        run(q, kp, vp, ko, vo, 100, 10, 109)       # score rows shorter than the context
    with pytest.raises(ValueError):
        run(q, kp.transpose(0, 1).contiguous(), vp, ko, vo, 100, 10)
    with pytest.raises(E.EmblaError):
        run(q, kp, vp, ko, vo, 100, 10, alpha=0.0)
