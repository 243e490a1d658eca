"""Ragged window decode of NaN and infinite rows, in every form that the call takes: what a head's scores and a
ring's values make of them."""
import math

import pytest
import torch

import ragged_reference as R
import relu_sparse_kv_gb300 as E

pytestmark = pytest.mark.gpu

D = 128
DEV = "cuda"

# sequences, KV heads, group, ring: one CTA to a unit; clusters of 2, 4 and 8 that fit the SMs; rows gone through by
# four, two and one CTAs to a unit
FORMS = [(2, 4, 4, 128), (2, 2, 8, 100), (4, 4, 4, 256), (70, 2, 8, 200), (5, 4, 4, 300), (12, 2, 8, 512), (2, 4, 4, 1024),
         (12, 4, 4, 1000), (22, 4, 4, 1024), (50, 4, 4, 1024), (125, 2, 8, 1024), (260, 1, 4, 200)]


def _inputs(B, Hkv, G, W):
    gen = torch.Generator(device=DEV).manual_seed(B + W)
    draw = lambda *shape: torch.randn(*shape, generator=gen, device=DEV).bfloat16()
    # the first ones full; then none, one, two, a block of rows, half a ring
    pos = [2 * W, W - 1] + [(-1, 0, 1, 15, 16, W // 2, 3 * W)[b % 7] for b in range(2, B)]
    return draw(B, G * Hkv, D), draw(B, Hkv, W, D), draw(B, Hkv, W, D), pos


def _run(q, k, v, pos):
    B, Hkv, W, _ = k.shape
    out = torch.full((B, q.shape[1], D), 7.0, device=DEV)
    E.embla_window_decode_ragged(E.Shape(B, q.shape[1], Hkv, D, 0, 0), q, k, v,
                                 torch.tensor(pos, dtype=torch.int32, device=DEV), out)
    torch.cuda.synchronize()
    assert E.embla_device_check() == 0
    return out


def _rows(pos, W):
    return [min(p + 1, W) for p in pos]


@pytest.mark.parametrize("B,Hkv,G,W", FORMS)
def test_a_nan_in_a_query_makes_its_head_nan(B, Hkv, G, W):
    q, k, v, pos = _inputs(B, Hkv, G, W)
    want, tol = R.window_decode(q, k, v, pos, D ** -0.5)
    broken = torch.zeros(B, G * Hkv, dtype=torch.bool, device=DEV)
    for b in range(B):
        h = (5 * b) % (G * Hkv)
        q[b, h, 3 * b % D] = math.nan
        broken[b, h] = pos[b] >= 0  # (without keys nothing is computed from it)
    out = _run(q, k, v, pos)
    assert torch.isnan(out[broken]).all()
    R.assert_within(out[~broken], want[~broken], tol[~broken], "the other heads")


@pytest.mark.parametrize("rows", ["first", "last", "sixteen", "share", "all"])
@pytest.mark.parametrize("B,Hkv,G,W", FORMS)
def test_nan_keys_make_their_heads_nan(B, Hkv, G, W, rows):
    """One KV head of each sequence has them; as many as a warp or a CTA may have to itself."""
    q, k, v, pos = _inputs(B, Hkv, G, W)
    want, tol = R.window_decode(q, k, v, pos, D ** -0.5)
    broken = torch.zeros(B, Hkv, dtype=torch.bool, device=DEV)
    for b, n in enumerate(_rows(pos, W)):
        g = b % Hkv
        lo, hi = {"first": (0, 1), "last": (max(n - 1, 0), n), "sixteen": (0, min(n, 16)), "share": (max(0, n - 128), n),
                  "all": (0, n)}[rows]
        k[b, g, lo:hi, 17] = math.nan
        broken[b, g] = n > 0
    out = _run(q, k, v, pos)
    broken = broken.repeat_interleave(G, 1)
    assert torch.isnan(out[broken]).all()
    R.assert_within(out[~broken], want[~broken], tol[~broken], "the other heads")


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("B,Hkv,G,W", FORMS)
def test_a_broken_value_reaches_its_column(B, Hkv, G, W, value):
    """The column of a value that is infinite or NaN takes that value in every head of its group, whatever the
    weights; with infinities of both signs it is NaN."""
    q, k, v, pos = _inputs(B, Hkv, G, W)
    clean = v.clone()
    expect = torch.zeros(B, Hkv, D, dtype=torch.float64, device=DEV)
    for b, n in enumerate(_rows(pos, W)):
        for g in range(Hkv):
            for col, at in ((3, [0]), (70, [n - 1]), (90, [0, n // 2])):
                for i, j in enumerate(at):
                    x = -value if i else value
                    if n > 0:
                        v[b, g, j, col], clean[b, g, j, col] = x, 0.0
                        expect[b, g, col] += x if n > 1 or not i else -x
                    if n == 1:
                        v[b, g, 0, col], expect[b, g, col] = value, value
    want, tol = R.window_decode(q, k, clean, pos, D ** -0.5)
    expect = expect.repeat_interleave(G, 1)
    out = _run(q, k, v, pos).double()
    finite = torch.isfinite(expect)
    R.assert_within(out[finite], want[finite], tol[finite], "the other columns")
    got, x = out[~finite], expect[~finite]
    assert ((got == x) | (torch.isnan(got) & torch.isnan(x))).all()


@pytest.mark.parametrize("B,Hkv,G,W", FORMS)
def test_weights_that_vanish(B, Hkv, G, W):
    """A key whose weight is too small for a float still passes an infinite value on; one whose score is minus infinity
    contributes nothing."""
    q, k, v, pos = _inputs(B, Hkv, G, W)
    q[..., 0], k[..., 0] = 64.0, 0.0
    clean, low = v.clone(), k.clone()
    rows = _rows(pos, W)
    for b, n in enumerate(rows):
        if n > 1:
            k[b, :, 1, 0] = low[b, :, 1, 0] = -64.0  # tau 64^2 = 362 below the others
            v[b, :, 1, 5], clean[b, :, 1, 5] = math.inf, 0.0
        if n > 2:
            k[b, :, n - 1, 0], low[b, :, n - 1, 0] = -math.inf, -128.0  # (weighs less than 64 bits tell from nothing)
            v[b, :, n - 1, 9], clean[b, :, n - 1, 9] = math.nan, 0.0
    want, tol = R.window_decode(q, low, clean, pos, D ** -0.5)
    out = _run(q, k, v, pos)
    hit = torch.zeros(out.shape, dtype=torch.bool, device=DEV)
    hit[[b for b, n in enumerate(rows) if n > 1], :, 5] = True
    assert (out[hit] == math.inf).all()
    R.assert_within(out[~hit], want[~hit], tol[~hit], "the rest")


@pytest.mark.parametrize("B,Hkv,G,W", FORMS)
def test_values_whose_sum_overflows(B, Hkv, G, W):
    """The mean of values near the largest finite one is finite, though their sum is not."""
    q, k, v, pos = _inputs(B, Hkv, G, W)
    v.copy_((3e38 * torch.sign(v.float())).bfloat16())
    v[..., :40] = 3e38
    out = _run(q, k, v, pos)
    assert torch.isfinite(out).all()
    R.assert_within(out, *R.window_decode(q, k, v, pos, D ** -0.5), "large values")
