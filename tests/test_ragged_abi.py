"""CPU-side checks of the calls on packed sequences of different lengths: what they refuse before
touching the device, what is a no-op, and the block numbers that the attention kernel walks."""
import ctypes
import random

import pytest
import torch

import relu_sparse_kv_gb300 as E
from relu_sparse_kv_gb300 import build as B

OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA = 0, 1, 2, 3, 4
A = [ctypes.c_void_p(256 * (k + 1)) for k in range(16)]  # aligned, never dereferenced
ODD = ctypes.c_void_p(264)                               # 8-byte aligned only
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    B.build()
    return E.library()


def _shape(**kw):
    d = dict(batch=3, n_q_heads=16, n_kv_heads=4, head_dim=128, ctx_len=0, cache_stride=0)
    d.update(kw)
    return ctypes.byref(E._Shape(**d))


SHAPES = [(dict(head_dim=64), UNSUPPORTED), (dict(n_q_heads=12), UNSUPPORTED), (dict(n_kv_heads=3), INVALID),
          (dict(batch=-1), INVALID), (dict(n_kv_heads=0), INVALID)]


def _rope(lib, shape=None, T=100, cu=A[0], pos0=A[1], q=A[2], qs=2048, k=A[3], ks=512, v=A[4], vs=512, base=1e4,
          norm=0, eps=1e-6, qg=None, kg=None, qo=A[5], ko=A[6], window=128, kw=A[7], vw=A[8]):
    return lib.embla_rope_qkv(shape or _shape(), T, cu, pos0, q, qs, k, ks, v, vs, base, norm, eps, qg, kg, qo, ko,
                              window, kw, vw, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(cu=None), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(qo=None), INVALID), (dict(kw=None), INVALID), (dict(vw=None), INVALID),
    (dict(qs=2040), INVALID), (dict(qs=2052), INVALID), (dict(ks=508), INVALID), (dict(vs=0), INVALID),
    (dict(base=0.0), INVALID), (dict(base=-1.0), INVALID), (dict(base=INF), INVALID), (dict(base=NAN), INVALID),
    (dict(norm=1, eps=-1.0), INVALID), (dict(norm=1, eps=NAN), INVALID), (dict(qg=A[9]), INVALID),
    (dict(kg=A[9]), INVALID), (dict(window=0), INVALID), (dict(window=1025), INVALID),
    (dict(T=(1 << 30) + 1), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED), (dict(qs=1 << 40), UNSUPPORTED),
    *[({name: ODD}, INVALID) for name in ("cu", "pos0", "q", "k", "v", "qo", "ko", "kw", "vw")],
    (dict(norm=1, qg=ODD), INVALID), (dict(norm=1, kg=ODD), INVALID),
])
def test_rope_refusals(lib, kw, status):
    assert _rope(lib, **kw) == status


def test_rope_no_ops(lib):
    assert _rope(lib, T=0, cu=None, q=None, k=None, v=None, qo=None) == OK
    assert _rope(lib, shape=_shape(batch=0)) == OK
    for kw, status in SHAPES:
        assert _rope(lib, shape=_shape(**kw)) == status
    assert lib.embla_rope_qkv(None, 0, *[None] * 3, 0, None, 0, None, 0, 1e4, 0, 0.0, *[None] * 4, 0, None, None,
                              None) == INVALID


def _window(lib, shape=None, T=100, cu=A[0], N=100, cuk=None, q=A[2], qs=2048, k=A[3], ks=512, v=A[4], vs=512,
            window=128, tau=0.1, out=A[5]):
    return lib.embla_window_prefill(shape or _shape(), T, cu, N, cuk, q, qs, k, ks, v, vs, window, tau, out, None)


def _packed(lib, shape=None, T=100, cu=A[0], N=100, cuk=None, q=A[2], qs=2048, k=A[3], ks=512, v=A[4], vs=512,
            alpha=1.0, c=1.0, eps=1e-6, out=A[5], ws=A[6], wsb=1 << 30):
    return lib.embla_prefill_packed(shape or _shape(), T, cu, N, cuk, q, qs, k, ks, v, vs, alpha, c, eps, out, ws,
                                    wsb, None)


BOTH = [
    (dict(T=-1, N=-1), INVALID), (dict(N=-1, cuk=A[7]), INVALID), (dict(N=101), INVALID), (dict(cu=None), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(out=None), INVALID),
    (dict(qs=2040), INVALID), (dict(ks=516), INVALID), (dict(vs=-512), INVALID),
    (dict(T=(1 << 30) + 1, N=(1 << 30) + 1), UNSUPPORTED), (dict(N=1 << 30, cuk=A[7]), UNSUPPORTED),
    (dict(ks=1 << 40), UNSUPPORTED),
    *[({name: ODD}, INVALID) for name in ("cu", "cuk", "q", "k", "v", "out")],
]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(window=0), INVALID), (dict(window=-5), INVALID), (dict(tau=NAN), INVALID), (dict(tau=INF), INVALID)])
def test_window_prefill_refusals(lib, kw, status):
    assert _window(lib, **kw) == status


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(alpha=0.0), INVALID), (dict(alpha=INF), INVALID), (dict(c=-1.0), INVALID), (dict(eps=NAN), INVALID),
    (dict(ws=None), INVALID), (dict(ws=ODD), INVALID), (dict(wsb=1000), WORKSPACE)])
def test_prefill_packed_refusals(lib, kw, status):
    assert _packed(lib, **kw) == status


def test_packed_no_ops_and_sizes(lib):
    for f in (_window, _packed):
        assert f(lib, T=0, N=0, cu=None, q=None, k=None, v=None, out=None) == OK
        assert f(lib, T=0, N=50, cuk=A[7], q=None, out=None) == OK
        assert f(lib, shape=_shape(batch=0)) == OK
        for kw, status in SHAPES:
            assert f(lib, shape=_shape(**kw)) == status
    size = lib.embla_prefill_packed_workspace_size
    assert size(_shape(), 0) == 0 and size(_shape(head_dim=64), 10) == 0 and size(_shape(), -1) == 0
    for n in (1, 3, 4, 127, 5000):
        # every key's norm per KV head, and a tile past the last
        assert size(_shape(), n) >= 4 * (4 * n + 128)


def _decode(lib, shape=None, q=A[0], k=A[1], v=A[2], window=128, pos=A[3], tau=0.1, out=A[4]):
    return lib.embla_window_decode_ragged(shape or _shape(), q, k, v, window, pos, tau, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(window=0), INVALID), (dict(window=1025), INVALID), (dict(tau=NAN), INVALID), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(pos=None), INVALID), (dict(out=None), INVALID),
    *[({name: ODD}, INVALID) for name in ("q", "k", "v", "pos", "out")],
    (dict(shape=_shape(batch=0), q=None), OK)] + [(dict(shape=_shape(**kw)), st) for kw, st in SHAPES])
def test_window_decode_ragged_refusals(lib, kw, status):
    assert _decode(lib, **kw) == status


def test_packed_calls_refuse_more_than_a_billion_sequences(lib):
    """(the searches' steps stay below 2^31)"""
    many = dict(batch=(1 << 30) + 1, n_q_heads=4, n_kv_heads=1)
    for call in (_rope, _window, _packed):
        assert call(lib, shape=_shape(**many)) == UNSUPPORTED


@pytest.mark.parametrize("R", [16, 32])
def test_block_numbers_cover_every_token_once(R):
    """Sequence b owns the numbers from floor(cu[b] / R) + b: every token of every sequence lies in exactly
    one block, all numbers lie below tokens / R + batch, and the search finds the owner."""
    rng = random.Random(R)
    for _ in range(60):
        batch = rng.randrange(1, 90)
        lens = [rng.choice([0, 1, rng.randrange(R + 1), rng.randrange(5 * R), R, 4 * R]) for _ in range(batch)]
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        tokens = cu[-1] + rng.choice([0, 1, 3 * R])  # rows behind the last sequence
        seen = [0] * tokens
        for v in range(tokens // R + batch):
            lo, hi = 0, batch
            while hi > lo:  # as the kernel searches: 32 lanes look at once
                step = (hi - lo + 31) // 32
                ats = [lo + (lane + 1) * step for lane in range(32)]
                n = sum(at <= hi and cu[at] // R + at <= v for at in ats)
                lo, hi = lo + n * step, min(hi, lo + n * step + step - 1)
            assert lo == max(b for b in range(batch + 1) if cu[b] // R + b <= v)
            if lo == batch:
                continue
            t0 = (v - (cu[lo] // R + lo)) * R
            for t in range(t0, min(t0 + R, lens[lo])):
                seen[cu[lo] + t] += 1
        assert seen == [1] * cu[-1] + [0] * (tokens - cu[-1])


def test_binding_refuses_what_the_calls_cannot_read():
    shape = E.Shape(2, 16, 4, 128, 0, 0)
    cu = torch.tensor([0, 3, 5], dtype=torch.int32)
    q, k = torch.zeros(5, 16, 128, dtype=torch.bfloat16), torch.zeros(5, 4, 128, dtype=torch.bfloat16)
    out = torch.zeros_like(q)
    for call in (E.embla_window_prefill, E.embla_prefill_packed):
        with pytest.raises(ValueError):   # not on a GPU
            call(shape, cu, q, k, k, out)
        with pytest.raises(ValueError):   # one KV head short
            call(shape, cu, q, k[:, :3], k, out)
    with pytest.raises(ValueError):
        E.embla_rope_qkv(shape, cu, None, q, k, k, out, None)
    with pytest.raises(ValueError):
        E.embla_window_decode_ragged(shape, q[:2], None, None, cu[:2], out[:2].float())
