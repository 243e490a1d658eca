"""Rows of extreme sizes through the calls on packed prompts, and the calls on a stream of the caller's."""
import math

import pytest
import torch

import ragged_reference as R
import relu_sparse_kv_gb300 as E

pytestmark = pytest.mark.gpu

D = 128
DEV = "cuda"


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _bf(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV).bfloat16()


def _cu(lens):
    return torch.tensor(R.starts(lens), dtype=torch.int32, device=DEV)


def _checked():
    torch.cuda.synchronize()
    assert E.embla_device_check() == 0


@pytest.mark.parametrize("behind", [0, 5000])  # (many rows behind: the form for long contexts)
@pytest.mark.parametrize("Hkv,G", [(4, 4), (2, 8)])
@pytest.mark.parametrize("q_size,k_size,c,eps", [(57, 0, 1.0, 1e-6), (59, 0, 1.0, 0.0), (59, 40, 0.0, 1e-6), (59, -40, 1.0, 0.0),
                                                 (-48, 0, 0.0, 0.0), (-48, 40, 1.0, 0.0), (59, 59, 1.0, 0.0),
                                                 (-48, -48, 0.0, 0.0)])
def test_full_layers_do_not_ask_how_long_the_rows_are(Hkv, G, q_size, k_size, c, eps, behind):
    """Rows of q and k are normalised, so powers of two before them change nothing; the squares of scores before the
    query's norm need not fit a float."""
    lens = [300, 1, 77]
    gen, n, at = _gen(60), sum(lens), R.starts(lens)
    q, k, v = _bf(gen, n + behind, G * Hkv, D), _bf(gen, n + behind, Hkv, D), _bf(gen, n + behind, Hkv, D)
    q[::3] *= 2.0 ** q_size
    k[::2] *= 2.0 ** k_size
    out = torch.full_like(q, 7.0)
    E.embla_prefill_packed(E.Shape(3, G * Hkv, Hkv, D, 0, 0), _cu(lens), q, k, v, out, c=c, eps=eps)
    _checked()
    R.assert_within(out[:n], *R.prefill_packed(q[:n], k[:n], v[:n], at, at, 1.0, c, eps), "long and short rows")
    assert (out[n:] == 7.0).all()


@pytest.mark.parametrize("window", [1, 100, 1 << 30])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [10, 14, 16, 20, 40, 60])
@pytest.mark.parametrize("n", [100, 300])
def test_window_prefill_of_scores_far_from_zero(n, size, sign, window):
    """Scores that fp32 holds exactly, tau q . k = sign 2^(2 size - 3) (1 + r / 128): the largest ones take all of the
    weight where their distance from the next does, also where the scores' own unit in the last place is more than the
    exponential can reach.  (Tolerance: weights and outputs rounded to bf16; the exponents, tau log2(e) (s - max), are
    off by 2^-22 of the distance, and a weight counts below 150 of them.)"""
    Hkv, G = 2, 8
    q = torch.zeros(n, G * Hkv, D, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(n, Hkv, D, dtype=torch.bfloat16, device=DEV)
    v = _bf(_gen(61), n, Hkv, D)
    r = (torch.arange(n, device=DEV) * 37) % 128
    q[..., 5] = sign * 2.0 ** size
    k[..., 5] = (2.0 ** size * (1 + r[:, None] / 128)).bfloat16()
    out = torch.full_like(q, 7.0)
    E.embla_window_prefill(E.Shape(1, G * Hkv, Hkv, D, 0, 0), _cu([n]), q, k, v, out, window=window, tau=0.125)
    _checked()
    want, _ = R.window_prefill(q, k, v, [0, n], [0, n], window, 0.125)
    mean, _ = R.window_prefill(q, k, v.abs(), [0, n], [0, n], window, 0.125)
    R.assert_within(out, want, R.BF16 * want.abs() + (R.BF16 + 150 * 2.0 ** -22) * mean * 1.02, f"scores of 2^{2 * size - 3}")


@pytest.mark.parametrize("eps", [0.0, 1e-5])
@pytest.mark.parametrize("Hkv,G", [(4, 4), (2, 8)])
def test_rotation_norms_long_and_short_rows(Hkv, G, eps):
    """Rows whose root mean square lies between 2^-48 and 2^59, as the call is defined for."""
    gen, n = _gen(62), 160
    shape = E.Shape(1, G * Hkv, Hkv, D, 0, 0)
    q, k = _bf(gen, n, G * Hkv, D), _bf(gen, n, Hkv, D)
    sizes = torch.tensor([-47, -46, -45, -44, -40, -30, -20, -8, 0, 0, 9, 17, 30, 45, 57, 58], device=DEV)
    turn = torch.arange(n, device=DEV)[:, None]
    for x in (q, k):
        x.mul_(torch.pow(2.0, sizes[(turn + torch.arange(x.shape[1], device=DEV)) % 16].double())[..., None].float())
    qg, kg = (1 + 0.3 * torch.randn(D, generator=gen, device=DEV) for _ in range(2))
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    E.embla_rope_qkv(shape, _cu([n]), None, q, k, None, q_out, k_out, norm_eps=eps, q_gain=qg, k_gain=kg)
    _checked()
    pos = torch.arange(n, device=DEV)
    for got, x, g, what in ((q_out, q, qg, "q_out"), (k_out, k, kg, "k_out")):
        want, tol = R.rope(x, pos, 10000.0, g, eps)
        R.assert_within(got, want, tol, what)


def test_rope_and_decode_on_a_stream_of_the_caller():
    """A rotation into the rings, and a decode that reads them, on a stream that is busy when they are called: both
    wait for what is before them there, and what they write is the reference's."""
    gen = _gen(63)
    lens, first, Hkv, W = [1, 30, 7], [5, 3, 100], 4, 16
    B, n, at = len(lens), sum(lens), R.starts(lens)
    shape, cu = E.Shape(B, 16, Hkv, D, 0, 0), _cu(lens)
    pos0 = torch.tensor(first, dtype=torch.int32, device=DEV)
    last = [f + m - 1 for f, m in zip(first, lens)]
    pos1 = torch.tensor(last, dtype=torch.int32, device=DEV)
    q, k, v, qb = _bf(gen, n, 16, D), _bf(gen, n, Hkv, D), _bf(gen, n, Hkv, D), _bf(gen, B, 16, D)
    late = [torch.zeros_like(x) for x in (q, k, v)]
    old = [_bf(gen, B, Hkv, W, D) for _ in range(2)]
    rings = [torch.zeros_like(x) for x in old]
    q_out, k_out, out = torch.zeros_like(q), torch.zeros_like(k), torch.full((B, 16, D), 7.0, device=DEV)
    busy = torch.zeros(1 << 28, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(8):
            busy.add_(1.0)
        for to, x in zip(late + rings, [q, k, v] + old):
            to.copy_(x)
    E.embla_rope_qkv(shape, cu, pos0, *late, q_out, k_out, k_win=rings[0], v_win=rings[1], stream=side)
    E.embla_window_decode_ragged(shape, qb, *rings, pos1, out, stream=side)
    _checked()
    pos = torch.cat([torch.arange(f, f + m, device=DEV) for f, m in zip(first, lens)])
    R.assert_within(q_out, *R.rope(q, pos, 10000.0), "queries")
    R.assert_within(k_out, *R.rope(k, pos, 10000.0), "keys")
    for b, m in enumerate(lens):
        for t in range(max(0, m - W), m):
            old[0][b, :, (first[b] + t) % W], old[1][b, :, (first[b] + t) % W] = k_out[at[b] + t], v[at[b] + t]
    assert torch.equal(rings[0], old[0]) and torch.equal(rings[1], old[1])
    R.assert_within(out, *R.window_decode(qb, *old, last, D ** -0.5), "decode")
