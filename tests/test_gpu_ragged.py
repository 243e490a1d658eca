"""Packed prompts of different lengths and the step after them on the GPU: rotation, window attention, full
layers, ragged window decode, each against a plain 64-bit form, and a run of them together."""
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


def _bf(gen, *shape, scale=1.0):
    return (scale * torch.randn(*shape, generator=gen, device=DEV)).bfloat16()


def _cu(lens):
    return torch.tensor(R.starts(lens), dtype=torch.int32, device=DEV)


def _checked():
    torch.cuda.synchronize()
    assert E.embla_device_check() == 0


def _fused(gen, T, Hq, Hkv, pad=0):
    """q, k, v as parts of one projection's rows, `pad` elements between tokens."""
    x = _bf(gen, T, (Hq + 2 * Hkv) * D + pad)[:, :(Hq + 2 * Hkv) * D].unflatten(1, (Hq + 2 * Hkv, D))
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


# ----------------------------------------------------------------------------- rotation

@pytest.mark.parametrize("lens,Hkv,pos0,norm,window", [
    ([1], 4, [0], False, 128),
    ([1] * 8, 4, [0, 1, 127, 128, 32768, 131071, 1 << 20, 2_000_000_000], False, 128),
    ([5, 0, 300, 1, 128, 129, 127], 2, None, True, 128),
    ([700, 33], 4, [100, 99999], True, 1024),
    ([40, 0, 0, 7] * 20, 2, [3 * i for i in range(80)], False, 16),  # more sequences than one step of the search
    ([1000], 1, [50], True, 1),
    ([64, 65], 8, [0, 7], False, 100),
])
def test_rope(lens, Hkv, pos0, norm, window):
    gen = _gen(sum(lens) + Hkv)
    G = 8 if Hkv <= 2 else 4
    Hq, B, T = G * Hkv, len(lens), sum(lens)
    behind = 9
    q, k, v = _fused(gen, T + behind, Hq, Hkv, pad=24)
    qg = 1 + 0.3 * torch.randn(D, generator=gen, device=DEV) if norm else None
    kg = 1 + 0.3 * torch.randn(D, generator=gen, device=DEV) if norm else None
    eps = 1e-5 if norm else None
    q_out = torch.full((T + behind, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    k_out = torch.full((T + behind, Hkv, D), 7.0, dtype=torch.bfloat16, device=DEV)
    k_win = torch.full((B, Hkv, window, D), 5.0, dtype=torch.bfloat16, device=DEV)
    v_win = torch.full((B, Hkv, window, D), 5.0, dtype=torch.bfloat16, device=DEV)
    cu = _cu(lens)
    p0 = None if pos0 is None else torch.tensor(pos0, dtype=torch.int32, device=DEV)
    E.embla_rope_qkv(E.Shape(B, Hq, Hkv, D, 0, 0), cu, p0, q, k, v, q_out, k_out, norm_eps=eps, q_gain=qg, k_gain=kg,
                     k_win=k_win, v_win=v_win)
    _checked()
    pos = torch.cat([torch.arange(n, device=DEV) + (0 if pos0 is None else pos0[b]) for b, n in enumerate(lens)])
    for got, x, g, what in ((q_out, q, qg, "q_out"), (k_out, k, kg, "k_out")):
        R.assert_within(got[:T], *R.rope(x[:T], pos, 10000.0, g, eps), what)
        assert (got[T:] == 7.0).all(), "rows behind the last sequence"
    kw, vw = torch.full_like(k_win, 5.0), torch.full_like(v_win, 5.0)
    at = R.starts(lens)
    for b, n in enumerate(lens):
        for t in range(at[b] + max(0, n - window), at[b] + n):
            kw[b, :, int(pos[t]) % window], vw[b, :, int(pos[t]) % window] = k_out[t], v[t]
    assert torch.equal(k_win, kw) and torch.equal(v_win, vw)


def test_rope_in_place_without_rings_and_nan():
    gen = _gen(3)
    shape = E.Shape(2, 16, 4, D, 0, 0)
    cu = _cu([100, 61])
    q, k = _bf(gen, 161, 16, D), _bf(gen, 161, 4, D)
    q[50, 3, 17] = math.nan
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    E.embla_rope_qkv(shape, cu, None, q, k, None, q_out, k_out, norm_eps=0.0)
    broken = torch.isnan(q_out).any(-1)
    assert broken.nonzero().tolist() == [[50, 3]]  # the row of the NaN alone
    only_q = torch.empty_like(q)
    E.embla_rope_qkv(shape, cu, None, q, k, None, only_q, None, norm_eps=0.0)
    E.embla_rope_qkv(shape, cu, None, q, k, None, q, k, norm_eps=0.0)
    _checked()
    for a, b in ((q, q_out), (only_q, q_out), (k, k_out)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


# ----------------------------------------------------------------------------- attention

LENS = [
    ([1], None), ([7], None), ([32], None), ([33, 1, 0, 31], None), ([16, 17, 15, 128, 129, 127], None),
    ([300, 1, 0, 0, 511], None), ([1000], None), ([2, 0, 5] * 30, None),
    ([5, 40, 1, 0, 64], [700, 40, 300, 9, 65]),  # queries are the last of more keys
    ([9, 200, 3], [4, 0, 3]),                    # and of fewer: the first ones see nothing
    ([600, 0], [1300, 0]),
]


def _attention_inputs(seed, lens, klens, Hkv, G, behind, spread):
    gen = _gen(seed)
    T, N = sum(lens) + behind, (sum(lens) if klens is None else sum(klens)) + behind
    if klens is None:
        q, k, v = _fused(gen, T, G * Hkv, Hkv, pad=8)
    else:
        q = _bf(gen, T, G * Hkv, D)
        _, k, v = _fused(gen, N, G * Hkv, Hkv)
    q.mul_(spread)
    out = torch.full((T, G * Hkv, D), 7.0, dtype=torch.bfloat16, device=DEV)
    return q, k, v, out


def _run_window(lens, klens, Hkv, q, k, v, out, window, tau=None, **kw):
    shape = E.Shape(len(lens), q.shape[1], Hkv, D, 0, 0)
    E.embla_window_prefill(shape, _cu(lens), q, k, v, out, window=window, tau=tau,
                           cu_keys=None if klens is None else _cu(klens), **kw)


def _run_packed(lens, klens, Hkv, q, k, v, out, **kw):
    shape = E.Shape(len(lens), q.shape[1], Hkv, D, 0, 0)
    E.embla_prefill_packed(shape, _cu(lens), q, k, v, out, cu_keys=None if klens is None else _cu(klens), **kw)


@pytest.mark.parametrize("window", [1, 2, 128, 200, 1024, 1 << 40])
@pytest.mark.parametrize("case", range(len(LENS)))
@pytest.mark.parametrize("Hkv,G", [(4, 4), (2, 8), (1, 4), (3, 8)])
def test_window_prefill(case, window, Hkv, G):
    if (Hkv in (1, 3)) != (window == 200):  # odd head counts at one window
        pytest.skip("covered")
    lens, klens = LENS[case]
    behind = 5 if case % 2 else 0
    q, k, v, out = _attention_inputs(case + window % 1000, lens, klens, Hkv, G, behind, 2.0)
    _run_window(lens, klens, Hkv, q, k, v, out, window)
    _checked()
    T = sum(lens)
    want, tol = R.window_prefill(q[:T], k, v, R.starts(lens), R.starts(klens or lens), window, D ** -0.5)
    R.assert_within(out[:T], want, tol, "window prefill")
    assert (out[T:] == 7.0).all(), "rows behind the last sequence"


@pytest.mark.parametrize("alpha,c,eps", [(1.0, 1.0, 1e-6), (0.3, 0.0, 1e-3)])
@pytest.mark.parametrize("case", range(len(LENS)))
@pytest.mark.parametrize("Hkv,G", [(4, 4), (2, 8), (3, 4)])
def test_prefill_packed(case, Hkv, G, alpha, c, eps):
    lens, klens = LENS[case]
    behind = 5 if case % 2 else 0
    q, k, v, out = _attention_inputs(case, lens, klens, Hkv, G, behind, 3.0)
    _run_packed(lens, klens, Hkv, q, k, v, out, alpha=alpha, c=c, eps=eps)
    _checked()
    T = sum(lens)
    want, tol = R.prefill_packed(q[:T], k, v, R.starts(lens), R.starts(klens or lens), alpha, c, eps)
    R.assert_within(out[:T], want, tol, "packed prefill")
    assert (out[T:] == 7.0).all(), "rows behind the last sequence"


@pytest.mark.parametrize("case", [c for c in range(len(LENS)) if len(LENS[c][0]) < 10])
@pytest.mark.parametrize("Hkv,G", [(4, 4), (2, 8), (3, 4)])
def test_prefill_packed_with_many_rows_behind(case, Hkv, G):
    """More rows than sequences fill have the call take the form for long ones; those rows hold NaN, and so
    do the values of some keys of weight zero."""
    lens, klens = LENS[case]
    q, k, v, out = _attention_inputs(40 + case, lens, klens, Hkv, G, 1600 * len(lens), 3.0)
    T, at = sum(lens), R.starts(klens or lens)
    k[at[-1]:] = math.nan
    v[at[-1]:] = math.inf
    k[10:at[-1]:37] = 0.0  # no direction: scores of zero
    clean = v[:at[-1]].clone()
    clean[10::37] = 0.0
    v[10:at[-1]:37] = math.nan
    _run_packed(lens, klens, Hkv, q, k, v, out)
    _checked()
    want, tol = R.prefill_packed(q[:T], k[:at[-1]], clean, R.starts(lens), at, 1.0, 1.0, 1e-6)
    R.assert_within(out[:T], want, tol, "rows behind")
    assert (out[T:] == 7.0).all()


def test_prefill_packed_equals_prefill_of_each():
    """The unpacked call, sequence by sequence, within both calls' precision."""
    lens, Hkv = [500, 129, 1, 258], 4
    q, k, v, out = _attention_inputs(8, lens, None, Hkv, 4, 0, 1.0)
    _run_packed(lens, None, Hkv, q, k, v, out)
    at = R.starts(lens)
    for a, b in zip(at, at[1:]):
        kc, vc = (x[a:b].transpose(0, 1).contiguous()[None] for x in (k, v))
        one = torch.empty(1, 16, b - a, D, device=DEV)
        E.embla_prefill(E.Shape(1, 16, Hkv, D, b - a, b - a), q[a:b].transpose(0, 1).contiguous()[None], kc, vc, one)
        want, tol = R.prefill_packed(q[a:b], k[a:b], v[a:b], [0, b - a], [0, b - a], 1.0, 1.0, 1e-6)
        R.assert_within(out[a:b], one[0].transpose(0, 1).double(), 2 * tol, "packed against unpacked")
    _checked()


@pytest.mark.parametrize("tau", [-0.3, 0.0, 1.5, 1e-4])
def test_window_prefill_scales(tau):
    lens = [200, 77]
    q, k, v, out = _attention_inputs(11, lens, None, 4, 4, 0, 1.0)
    _run_window(lens, None, 4, q, k, v, out, 100, tau=tau)
    _checked()
    R.assert_within(out, *R.window_prefill(q, k, v, R.starts(lens), R.starts(lens), 100, tau), f"tau {tau}")


@pytest.mark.parametrize("order", ["rising", "falling"])
def test_window_prefill_reference_follows_the_maximum(order):
    """Scores that rise along the context by far more than 2^8 a tile, and that fall again."""
    n, Hkv = 900, 4
    q, k, v, out = _attention_inputs(12, [n], None, Hkv, 4, 0, 1.0)
    u = torch.nn.functional.normalize(torch.randn(D, generator=_gen(1), device=DEV), dim=0)
    ramp = torch.arange(n, device=DEV) if order == "rising" else torch.arange(n, 0, -1, device=DEV)
    q.copy_(q.float() + 30 * u)
    k.copy_(k.float() + ramp[:, None, None] * u)
    _run_window([n], None, Hkv, q, k, v, out, 1 << 30)
    _checked()
    R.assert_within(out, *R.window_prefill(q, k, v, [0, n], [0, n], 1 << 30, D ** -0.5), order)


def _poison(x, rows, values):
    for i, r in enumerate(rows):
        x[r, :, (11 * i) % D] = values[i % len(values)]


@pytest.mark.parametrize("kind", ["window", "packed"])
def test_infinite_and_nan_rows_stay_where_they_are_seen(kind):
    """Rows that a query does not see, another sequence's or a later token's, may hold anything; the
    sequences beside a poisoned one and the tokens before it come out as if it were not there."""
    lens, Hkv, W = [60, 100, 45, 130], 4, 40
    at = R.starts(lens)
    q, k, v, out = _attention_inputs(13, lens, None, Hkv, 4, 3, 1.0)
    bad = [math.inf, math.nan, -math.inf]
    _poison(v, [at[1] + 70, at[1] + 71, at[3] + 129, at[4], at[4] + 2], bad)
    _poison(k, [at[1] + 72, at[4] + 1], [math.nan])
    run = (lambda o: _run_window(lens, None, Hkv, q, k, v, o, W)) if kind == "window" else \
        (lambda o: _run_packed(lens, None, Hkv, q, k, v, o))
    run(out)
    _checked()
    clean_k, clean_v = torch.nan_to_num(k, 0.0, 0.0, 0.0), torch.nan_to_num(v, 0.0, 0.0, 0.0)
    if kind == "window":
        want, tol = R.window_prefill(q[:at[4]], clean_k, clean_v, at, at, W, D ** -0.5)
        unseen = [t for t in range(at[4]) if not (at[1] + 70 <= t < min(at[2], at[1] + 72 + W)) and t != at[4] - 1]
    else:
        want, tol = R.prefill_packed(q[:at[4]], clean_k, clean_v, at, at, 1.0, 1.0, 1e-6)
        unseen = [t for t in range(at[4]) if not (at[1] + 70 <= t < at[2]) and t != at[4] - 1]
    R.assert_within(out[unseen], want[unseen], tol[unseen], "rows that see no poison")
    assert not torch.isfinite(out[at[1] + 71]).all()  # and those that see it show it


@pytest.mark.parametrize("behind", [0, 5000])  # (many rows behind: the full layers' form for long contexts)
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("Hkv,G", [(4, 4), (3, 8)])
def test_a_broken_value_reaches_one_column_of_the_rows_that_weigh_it(Hkv, G, value, behind):
    lens, W, col = [70, 300, 5], 100, 37
    n, at = sum(lens), R.starts(lens)
    q, k, v, window_out = _attention_inputs(50, lens, None, Hkv, G, behind, 1.0)
    full_out, clean = window_out.clone(), v.clone()
    broken = [(0, 69), (1, 0), (1, 150), (2, 2)]
    for b, j in broken:
        v[at[b] + j, :, col], clean[at[b] + j, :, col] = value, 0.0
    _run_window(lens, None, Hkv, q, k, v, window_out, W)
    _run_packed(lens, None, Hkv, q, k, v, full_out)
    _checked()
    others = [d for d in range(D) if d != col]
    for out, form in ((window_out, R.window_prefill(q[:n], k[:n], clean[:n], at, at, W, D ** -0.5)),
                      (full_out, R.prefill_packed(q[:n], k[:n], clean[:n], at, at, 1.0, 1.0, 1e-6))):
        want, tol = (x.expand(n, G * Hkv, D) for x in form)
        R.assert_within(out[:n][..., others], want[..., others], tol[..., others], "the other columns")
    unit = lambda x: x.double() / x.double().square().mean(-1, keepdim=True).sqrt()
    sees = torch.zeros(n, dtype=torch.bool, device=DEV)
    for b, j in broken:
        sees[at[b] + j:min(at[b + 1], at[b] + j + W)] = True
        dot = (unit(q[at[b] + j:at[b + 1]]) * unit(k[at[b] + j]).repeat_interleave(G, 0)).sum(-1)
        assert not torch.isfinite(full_out[at[b] + j:at[b + 1]][..., col])[dot > 0.1].any()
    finite = torch.isfinite(window_out[:n][..., col])
    assert finite[~sees].all() and not finite[sees].any()
    # one broken value: the rows of the other sign's scores do not weigh it
    dot = (unit(q[:70]) * unit(k[69]).repeat_interleave(G, 0)).sum(-1)
    assert torch.isfinite(full_out[:69][..., col]).all() and torch.isfinite(full_out[69][..., col])[dot[69] < -0.1].all()


@pytest.mark.parametrize("kind", ["window", "packed"])
@pytest.mark.parametrize("Hkv,G", [(4, 4), (2, 8)])
@pytest.mark.parametrize("before,n", [(0, 1), (1, 79), (2, 80), (3, 81), (130, 127), (5, 128), (7, 129), (38, 400)])
def test_a_sequence_among_nan_rows(kind, Hkv, G, before, n):
    """Every row of k and v but one sequence's is NaN or infinite, those behind the last sequence too."""
    lens = [before, n, 50]
    q, k, v, out = _attention_inputs(23 + n, lens, None, Hkv, G, 40, 1.0)
    for x, bad in ((k, math.nan), (v, math.inf)):
        x[:before] = bad
        x[before + n:] = -bad
    _run_window(lens, None, Hkv, q, k, v, out, 100) if kind == "window" else _run_packed(lens, None, Hkv, q, k, v, out)
    _checked()
    own = slice(before, before + n)
    form = R.window_prefill(q[own], k[own], v[own], [0, n], [0, n], 100, D ** -0.5) if kind == "window" else \
        R.prefill_packed(q[own], k[own], v[own], [0, n], [0, n], 1.0, 1.0, 1e-6)
    R.assert_within(out[own], *form, "the sequence between")
    assert (out[before + n + 50:] == 7.0).all()


@pytest.mark.parametrize("kind", ["window", "packed"])
def test_queries_without_any_key(kind):
    lens, Hkv = [3, 0, 40], 4
    q, k, v, out = _attention_inputs(24, lens, [0, 0, 0], Hkv, 4, 0, 1.0)
    assert k.shape[0] == 0
    _run_window(lens, [0, 0, 0], Hkv, q, k, v, out, 100) if kind == "window" else \
        _run_packed(lens, [0, 0, 0], Hkv, q, k, v, out)
    _checked()
    assert (out == 0.0).all()


def test_zero_weight_keys_hide_their_values():
    """ReLU^2: a key whose score is not positive, or NaN, weighs nothing even where its value is NaN."""
    n, Hkv = 200, 4
    q, k, v, out = _attention_inputs(14, [n], None, Hkv, 4, 0, 1.0)
    u = torch.nn.functional.normalize(torch.randn(D, generator=_gen(2), device=DEV), dim=0)
    q.copy_(0.1 * q.float() + 10 * u)
    k[50:60] = (-5 * u).bfloat16()
    k[61] = math.nan
    v[50:62] = math.nan
    k[60] = (-5 * u).bfloat16()
    _run_packed([n], None, Hkv, q, k, v, out)
    _checked()
    ck, cv = k.clone(), v.clone()
    ck[61] = (-5 * u).bfloat16()
    cv[50:62] = 0.0
    R.assert_within(out, *R.prefill_packed(q, ck, cv, [0, n], [0, n], 1.0, 1.0, 1e-6), "values of weight zero")


def test_rows_of_minus_infinite_scores_and_zero_queries():
    n, Hkv = 70, 4
    q, k, v, out = _attention_inputs(15, [n], None, Hkv, 4, 0, 1.0)
    q[10] = 0.0
    _run_window([n], None, Hkv, q, k, v, out, 30)
    R.assert_within(out, *R.window_prefill(q, k, v, [0, n], [0, n], 30, D ** -0.5), "a zero query: the mean")
    k[:, :, 0] = -math.inf
    q[:, :, 0] = 1.0
    _run_window([n], None, Hkv, q, k, v, out, 30)
    assert (out == 0.0).all()  # no key weighs anything
    q, k, v, out = _attention_inputs(16, [n], None, Hkv, 4, 0, 1.0)
    q[10] = 0.0
    _run_packed([n], None, Hkv, q, k, v, out, c=0.0)
    assert (out[10] == 0.0).all()
    _checked()


def test_outputs_on_16_bytes_and_large_values():
    lens, Hkv = [130, 20], 4
    q, k, v, _ = _attention_inputs(17, lens, None, Hkv, 4, 0, 1.0)
    v.mul_(2.0 ** 120)
    flat = torch.full((150 * 16 * D + 16,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = flat[8:8 + 150 * 16 * D].view(150, 16, D)
    assert out.data_ptr() % 32 == 16
    _run_window(lens, None, Hkv, q, k, v, out, 64)
    _checked()
    assert (flat[:8] == 7.0).all() and (flat[8 + 150 * 16 * D:] == 7.0).all()
    R.assert_within(out, *R.window_prefill(q, k, v, R.starts(lens), R.starts(lens), 64, D ** -0.5), "16-byte rows")


def test_values_whose_sum_overflows_before_it_is_divided():
    """A mean of values near the largest finite one is finite, though their sum is not."""
    n, Hkv = 160, 4
    q, k, v, out = _attention_inputs(18, [n], None, Hkv, 4, 0, 1.0)
    v.copy_((3e38 * torch.sign(v.float())).bfloat16())
    v[:, :, :64] = 3e38
    _run_window([n], None, Hkv, q, k, v, out, 128)
    _checked()
    assert torch.isfinite(out).all()
    R.assert_within(out, *R.window_prefill(q, k, v, [0, n], [0, n], 128, D ** -0.5), "large values")


@pytest.mark.parametrize("kind", ["window", "packed"])
def test_long_prompts_against_one_row_at_a_time(kind):
    """A few rows of prompts of thousands of tokens (many blocks per CTA, many tiles per block)."""
    lens, Hkv = [5000, 2500, 6100], 2
    at = R.starts(lens)
    q, k, v, out = _attention_inputs(19, lens, None, Hkv, 8, 0, 1.5)
    if kind == "window":
        _run_window(lens, None, Hkv, q, k, v, out, 1000)
    else:
        _run_packed(lens, None, Hkv, q, k, v, out)
    _checked()
    for b, n in enumerate(lens):
        for t in sorted({0, 1, 999, 1000, 1001, 2047, n - 17, n - 1}):
            a, e = at[b], at[b] + t
            if kind == "window":
                want, tol = R.window_prefill(q[e:e + 1], k[a:e + 1], v[a:e + 1], [0, 1], [0, t + 1], 1000, D ** -0.5)
            else:
                want, tol = R.prefill_packed(q[e:e + 1], k[a:e + 1], v[a:e + 1], [0, 1], [0, t + 1], 1.0, 1.0, 1e-6)
            R.assert_within(out[e:e + 1], want, tol, f"sequence {b} token {t}")


@pytest.mark.parametrize("kind", ["window", "packed"])
def test_sequences_that_do_not_ascend_are_reported(kind):
    """The first sequence's rows that no other entry claims come out as ever."""
    Hkv = 4
    q, k, v, out = _attention_inputs(20, [100], None, Hkv, 4, 0, 1.0)
    good = torch.full_like(out, 7.0)
    for cu in ([0, 40, 30, 100], [0, 40, 500, 100], [0, 40, -7, 60]):
        out.fill_(7.0)
        shape = E.Shape(3, 16, Hkv, D, 0, 0)
        cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
        if kind == "window":
            E.embla_window_prefill(shape, cut, q, k, v, out)
        else:
            E.embla_prefill_packed(shape, cut, q, k, v, out)
        torch.cuda.synchronize()
        assert E.embla_device_check() == 1
        (_run_window([40], None, Hkv, q[:40], k[:40], v[:40], good[:40], 128) if kind == "window" else
         _run_packed([40], None, Hkv, q[:40], k[:40], v[:40], good[:40]))
        assert torch.equal(out[:30], good[:30])
    assert E.embla_device_check() == 0


@pytest.mark.parametrize("kind", ["window", "packed"])
def test_graph_serves_other_lengths_and_streams_do_not_mix(kind):
    Hkv, T, B = 4, 400, 3
    shape = E.Shape(B, 16, Hkv, D, 0, 0)
    q, k, v, out = _attention_inputs(21, [T], None, Hkv, 4, 0, 1.0)
    cu = _cu([100, 200, 100])
    ws = torch.empty(E.embla_prefill_packed_workspace_size(shape, T), dtype=torch.uint8, device=DEV)

    def call(stream=None):
        if kind == "window":
            E.embla_window_prefill(shape, cu, q, k, v, out, window=90, stream=stream)
        else:
            E.embla_prefill_packed(shape, cu, q, k, v, out, workspace=ws, stream=stream)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([100, 200, 100], [0, 399, 1], [400, 0, 0], [5, 6, 7]):
        cu.copy_(_cu(lens))
        out.fill_(7.0)
        graph.replay()
        _checked()
        n = sum(lens)
        if kind == "window":
            want, tol = R.window_prefill(q[:n], k[:n], v[:n], R.starts(lens), R.starts(lens), 90, D ** -0.5)
        else:
            want, tol = R.prefill_packed(q[:n], k[:n], v[:n], R.starts(lens), R.starts(lens), 1.0, 1.0, 1e-6)
        R.assert_within(out[:n], want, tol, f"replayed with {lens}")
        assert (out[n:] == 7.0).all()
    first = out.clone()
    out.fill_(0.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    # a second call beside it, with outputs of its own
    other = torch.empty_like(out)
    (E.embla_window_prefill(shape, cu, q, k, v, other, window=90) if kind == "window" else
     E.embla_prefill_packed(shape, cu, q, k, v, other))
    torch.cuda.synchronize()
    assert torch.equal(out[:18], first[:18]) and torch.equal(other[:18], first[:18])


def test_attention_refuses_what_it_cannot_read():
    q, k, v, out = _attention_inputs(22, [10], None, 4, 4, 0, 1.0)
    shape, cu = E.Shape(1, 16, 4, D, 0, 0), _cu([10])
    for call in (E.embla_window_prefill, E.embla_prefill_packed):
        with pytest.raises(ValueError):
            call(shape, cu, q.transpose(0, 1).contiguous().transpose(0, 1), k, v, out)  # head-major rows
        with pytest.raises(ValueError):
            call(shape, cu, q, k[:9], v[:9], out)                                       # fewer keys, no cu_keys
        with pytest.raises(ValueError):
            call(shape, cu, q, k, v, out[:9])
        with pytest.raises(TypeError):
            call(shape, cu, q, k, v, out.float())
        with pytest.raises(TypeError):
            call(shape, cu.long(), q, k, v, out)
        with pytest.raises(ValueError):
            call(shape, _cu([4, 6]), q, k, v, out)                                      # another batch
    with pytest.raises(E.EmblaError) as err:
        E.embla_window_prefill(shape, cu, q, k, v, out, window=0)
    assert err.value.status == 1
    with pytest.raises(E.EmblaError) as err:
        E.embla_prefill_packed(shape, cu, q, k, v, out, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert err.value.status == 3


# ----------------------------------------------------------------------------- decode

@pytest.mark.parametrize("window", [1, 5, 128, 129, 300, 512, 700, 1024])
@pytest.mark.parametrize("Hkv,G", [(4, 4), (2, 8)])
def test_window_decode_ragged(window, Hkv, G):
    gen = _gen(window)
    pos = [0, -1, 1, 126, 127, 128, 255, 256, 511, window - 1, window, window + 13, 100000]
    B = len(pos)
    q = _bf(gen, B, G * Hkv, D, scale=2.0)
    k, v = _bf(gen, B, Hkv, window, D), _bf(gen, B, Hkv, window, D)
    for b, last in enumerate(pos):  # slots without a token hold anything
        if last + 1 < window:
            k[b, :, last + 1:], v[b, :, last + 1:] = math.nan, math.nan
    out = torch.full((B, G * Hkv, D), math.nan, device=DEV)
    E.embla_window_decode_ragged(E.Shape(B, G * Hkv, Hkv, D, 0, 0), q, k, v,
                                 torch.tensor(pos, dtype=torch.int32, device=DEV), out)
    _checked()
    R.assert_within(out, *R.window_decode(q, k, v, pos, D ** -0.5), "ragged window decode")


@pytest.mark.parametrize("B,Hkv,G,window", [(70, 4, 4, 1024), (120, 2, 8, 513), (130, 4, 4, 129), (230, 2, 8, 300)])
def test_window_decode_ragged_of_many_sequences(B, Hkv, G, window):
    """More sequences than fit the SMs one step each: longer shares, the running maximum rising and falling."""
    gen = _gen(B)
    pos = [(37 * b * b) % (2 * window) - 1 for b in range(B)]
    q = _bf(gen, B, G * Hkv, D, scale=2.0)
    k, v = _bf(gen, B, Hkv, window, D), _bf(gen, B, Hkv, window, D)
    u = torch.nn.functional.normalize(torch.randn(D, generator=gen, device=DEV), dim=0)
    ramp = torch.linspace(-3, 3, window, device=DEV)[:, None] * u
    q[::2] = (q[::2].float() + 10 * u).bfloat16()
    k[::4] = (k[::4].float() + ramp).bfloat16()
    k[2::4] = (k[2::4].float() - ramp).bfloat16()
    out = torch.full((B, G * Hkv, D), math.nan, device=DEV)
    E.embla_window_decode_ragged(E.Shape(B, G * Hkv, Hkv, D, 0, 0), q, k, v,
                                 torch.tensor(pos, dtype=torch.int32, device=DEV), out)
    _checked()
    R.assert_within(out, *R.window_decode(q, k, v, pos, D ** -0.5), "ragged window decode")


@pytest.mark.parametrize("B,Hkv,G,window", [(1, 1, 4, 128), (9, 4, 4, 128), (60, 4, 4, 128), (10, 2, 8, 300), (50, 2, 8, 300),
                                            (3, 4, 4, 1024), (200, 2, 8, 700)])
def test_window_decode_ragged_rows_that_hold_nothing_yet(B, Hkv, G, window):
    """NaN and infinities in the ring's unwritten rows, for batches of every form; nothing changes by them."""
    gen = _gen(window + B)
    pos = [(b * b * 7) % (window + 20) - 1 for b in range(B)]
    q, k, v = _bf(gen, B, G * Hkv, D), _bf(gen, B, Hkv, window, D), _bf(gen, B, Hkv, window, D)
    want = R.window_decode(q, k, v, pos, D ** -0.5)
    for b, p in enumerate(pos):
        k[b, :, max(0, p + 1):] = math.nan
        v[b, :, max(0, p + 1):] = -math.inf
    out = torch.full((B, G * Hkv, D), math.nan, device=DEV)
    E.embla_window_decode_ragged(E.Shape(B, G * Hkv, Hkv, D, 0, 0), q, k, v,
                                 torch.tensor(pos, dtype=torch.int32, device=DEV), out)
    _checked()
    R.assert_within(out, *want, "unwritten rows")


def test_window_decode_ragged_matches_window_decode():
    """All sequences at one position: the batch call with its own rotation of the query, and this one on
    the rotated query, agree within the rounding of that query to bf16 (2^-8 of each element, in the
    scores up to tau 2^-8 sum |q k|, twice in the weights)."""
    gen = _gen(4)
    B, Hkv, W, last = 5, 4, 128, 1000
    shape = E.Shape(B, 16, Hkv, D, 0, 0)
    q, k, v = _bf(gen, B, 16, D), _bf(gen, B, Hkv, W, D), _bf(gen, B, Hkv, W, D)
    one, two = torch.empty(B, 16, D, device=DEV), torch.empty(B, 16, D, device=DEV)
    E.embla_window_decode(shape, q, k, v, last, one)
    pos = torch.full((B,), last, dtype=torch.int32, device=DEV)
    turned = torch.empty_like(q)
    E.embla_rope_qkv(shape, _cu([1] * B), pos, q, q[:, :Hkv], None, turned, None)
    E.embla_window_decode_ragged(shape, turned, k, v, pos, two)
    _checked()
    size = torch.einsum("bhgd,bhjd->bhgj", turned.double().abs().view(B, Hkv, 4, D), k.double().abs()).amax(-1)
    err = 2 * D ** -0.5 * 2.0 ** -8 * size.reshape(B, 16, 1)
    _, tol = R.window_decode(turned, k, v, [last] * B, D ** -0.5)
    mean = v.double().abs().amax(2).repeat_interleave(4, 1)
    R.assert_within(two, one.double(), tol + err * mean, "against embla_window_decode")


def test_window_decode_ragged_graph_and_nan_rows():
    gen = _gen(6)
    B, Hkv, W = 4, 2, 300
    shape = E.Shape(B, 16, Hkv, D, 0, 0)
    q, k, v = _bf(gen, B, 16, D), _bf(gen, B, Hkv, W, D), _bf(gen, B, Hkv, W, D)
    pos = torch.tensor([0, 5, 200, 900], dtype=torch.int32, device=DEV)
    out = torch.empty(B, 16, D, device=DEV)
    E.embla_window_decode_ragged(shape, q, k, v, pos, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        E.embla_window_decode_ragged(shape, q, k, v, pos, out)
    for _ in range(3):
        pos += 1
        graph.replay()
        _checked()
        R.assert_within(out, *R.window_decode(q, k, v, pos.tolist(), D ** -0.5), "replayed at other positions")
    v[2, 0, 7, 9] = math.nan
    k[3, 1, 8] = math.nan
    graph.replay()
    _checked()
    broken = torch.isnan(out)
    assert broken[2, :8, 9].all() and broken[3, 8:].all() and int(broken.sum()) == 8 + 8 * D


# ----------------------------------------------------------------------------- calls

def test_offsets_past_32_bits():
    """Tokens 16 MB apart: rows lie past 2^32 bytes (and 2^32 elements) from the first."""
    lens, Hkv = [150, 0, 170], 2
    T, Hq, step = sum(lens), 16, 1 << 24
    x = torch.empty(T * step, dtype=torch.bfloat16, device=DEV)
    assert x.numel() > 1 << 32
    x = x.view(T, step)[:, :(Hq + 2 * Hkv) * D].unflatten(1, (Hq + 2 * Hkv, D))
    near = _bf(_gen(30), T, Hq + 2 * Hkv, D)
    x.copy_(near)
    shape, cu = E.Shape(3, Hq, Hkv, D, 0, 0), _cu(lens)
    parts = lambda y: (y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:])
    near[3, -1, 5] = x[3, -1, 5] = math.nan  # (a value row that makes its readers take the slow path)
    outs = []
    for y in (x, near):
        q, k, v = parts(y)
        out = [torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
        k_out = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV)
        rings = [torch.zeros(3, Hkv, 64, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        E.embla_window_prefill(shape, cu, q, k, v, out[0], window=70)
        E.embla_prefill_packed(shape, cu, q, k, v, out[1])
        E.embla_rope_qkv(shape, cu, None, q, k, v, out[2], k_out, k_win=rings[0], v_win=rings[1])
        _checked()
        outs.append([*out, k_out, *rings])
    for a, b in zip(*outs):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_rope_and_decode_on_a_stream_and_in_a_graph():
    """Positions and lengths are read as the graph runs; calls on another stream see what that stream wrote."""
    gen = _gen(31)
    B, Hkv, W = 3, 4, 16
    shape = E.Shape(B, 16, Hkv, D, 0, 0)
    q, k, v = _fused(gen, 12, 16, Hkv)
    cu, pos0 = _cu([4, 4, 4]), torch.tensor([0, 10, 30], dtype=torch.int32, device=DEV)
    last, qb = pos0 + 3, _bf(gen, B, 16, D)
    q_out, k_out = torch.zeros(12, 16, D, dtype=torch.bfloat16, device=DEV), torch.zeros(12, Hkv, D, dtype=torch.bfloat16, device=DEV)
    rings = [torch.zeros(B, Hkv, W, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    out = torch.zeros(B, 16, D, device=DEV)

    def step(stream=None):
        E.embla_rope_qkv(shape, cu, pos0, q, k, v, q_out, k_out, k_win=rings[0], v_win=rings[1], stream=stream)
        E.embla_window_decode_ragged(shape, qb, *rings, last, out, stream=stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens, first in (([4, 4, 4], [0, 10, 30]), ([1, 0, 11], [5, 3, 100]), ([12, 0, 0], [40, 0, 0])):
        cu.copy_(_cu(lens))
        pos0.copy_(torch.tensor(first, dtype=torch.int32))
        last.copy_(torch.tensor([f + n - 1 for f, n in zip(first, lens)], dtype=torch.int32))
        graph.replay()
        _checked()
        at = R.starts(lens)
        pos = torch.cat([torch.arange(f, f + n, device=DEV) for f, n in zip(first, lens)])
        R.assert_within(q_out, *R.rope(q, pos, 10000.0), "replayed queries")
        for b, n in enumerate(lens):
            for t in range(max(0, n - W), n):
                assert torch.equal(rings[0][b, :, (first[b] + t) % W], k_out[at[b] + t])
                assert torch.equal(rings[1][b, :, (first[b] + t) % W], v[at[b] + t])
        R.assert_within(out, *R.window_decode(qb, *rings, last.tolist(), D ** -0.5), "replayed decode")
    before = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q_out.zero_()
        out.zero_()
        for r in rings:
            r[:, :, 5:9] = 0.0
    step(stream=side)
    torch.cuda.synchronize()
    R.assert_within(q_out, *R.rope(q, pos, 10000.0), "on a stream")
    assert torch.isfinite(out).all() and out.shape == before.shape


def test_rope_refuses_what_it_cannot_read():
    gen = _gen(32)
    shape, cu = E.Shape(1, 16, 4, D, 0, 0), _cu([10])
    q, k, v = _fused(gen, 10, 16, 4)
    q_out, k_out = torch.empty(10, 16, D, dtype=torch.bfloat16, device=DEV), torch.empty(10, 4, D, dtype=torch.bfloat16, device=DEV)
    ring = torch.empty(1, 4, 8, D, dtype=torch.bfloat16, device=DEV)
    gain = torch.ones(D, device=DEV)
    for bad in (dict(q_out=q), dict(k=k[:9]), dict(k_win=ring), dict(v_win=ring), dict(k_win=ring[:, :, :0], v_win=ring[:, :, :0]),
                dict(pos0=cu), dict(k_win=ring, v_win=ring, v=v[:9])):
        args = dict(cu_tokens=cu, pos0=None, q=q, k=k, v=v, q_out=q_out, k_out=k_out) | bad
        with pytest.raises(ValueError):
            E.embla_rope_qkv(shape, **args)
    for bad in (dict(q_gain=gain), dict(norm_eps=-1.0), dict(rope_base=0.0)):
        with pytest.raises(E.EmblaError) as err:
            E.embla_rope_qkv(shape, cu, None, q, k, v, q_out, k_out, **bad)
        assert err.value.status == 1
    with pytest.raises(E.EmblaError) as err:
        E.embla_window_decode_ragged(shape, q_out[:1].contiguous(), torch.empty(1, 4, 1025, D, dtype=torch.bfloat16, device=DEV),
                                     torch.empty(1, 4, 1025, D, dtype=torch.bfloat16, device=DEV), cu[:1], torch.empty(1, 16, D, device=DEV))
    assert err.value.status == 1


@pytest.mark.parametrize("kind", ["window", "packed"])
def test_prompts_of_thousands_of_sequences(kind):
    """Many more sequences than CTAs, most of a token or none."""
    lens, Hkv = [(7 * b * b) % 5 if b % 97 else 300 for b in range(1500)], 2
    at = R.starts(lens)
    q, k, v, out = _attention_inputs(33, lens, None, Hkv, 8, 0, 1.5)
    _run_window(lens, None, Hkv, q, k, v, out, 128) if kind == "window" else _run_packed(lens, None, Hkv, q, k, v, out)
    _checked()
    some = [0, 1, 96, 97, 98, 700, 1455, 1499]
    for b in some:
        a, e = at[b], at[b + 1]
        form = R.window_prefill(q[a:e], k[a:e], v[a:e], [0, e - a], [0, e - a], 128, D ** -0.5) if kind == "window" else \
            R.prefill_packed(q[a:e], k[a:e], v[a:e], [0, e - a], [0, e - a], 1.0, 1.0, 1e-6)
        R.assert_within(out[a:e], *form, f"sequence {b}")


# ----------------------------------------------------------------------------- together

@pytest.mark.parametrize("Hkv,window", [(4, 128), (2, 40)])
def test_packed_prompts_then_steps(Hkv, window):
    """A window layer from packed prompts on, step by step: rotation into the rings, attention of the prompts, then
    one token per sequence at a time; every step is the row that a longer prompt would have had."""
    gen = _gen(Hkv)
    lens, steps = [150, 1, 39, 300], 3
    B, Hq = len(lens), 16
    full = [n + steps for n in lens]
    shape, at = E.Shape(B, Hq, Hkv, D, 0, 0), R.starts(full)
    x = _fused(gen, sum(full), Hq, Hkv)
    turned_q, turned_k, whole = (torch.empty(sum(full), h, D, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hq))
    E.embla_rope_qkv(shape, _cu(full), None, *x, turned_q, turned_k, norm_eps=1e-6)
    E.embla_window_prefill(shape, _cu(full), turned_q, turned_k, x[2], whole, window=window)
    prompt = torch.cat([torch.arange(at[b], at[b] + n, device=DEV) for b, n in enumerate(lens)])
    q, k, v = (y[prompt] for y in x)
    q_out, k_out, out = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
    rings = [torch.zeros(B, Hkv, window, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    E.embla_rope_qkv(shape, _cu(lens), None, q, k, v, q_out, k_out, norm_eps=1e-6, k_win=rings[0], v_win=rings[1])
    E.embla_window_prefill(shape, _cu(lens), q_out, k_out, v, out, window=window)
    assert torch.equal(q_out, turned_q[prompt])
    want, tol = R.window_prefill(turned_q, turned_k, x[2], at, at, window, D ** -0.5)
    R.assert_within(out, want[prompt], tol[prompt], "prompts")
    R.assert_within(whole, want, tol, "longer prompts")
    pos, cu1 = torch.tensor(lens, dtype=torch.int32, device=DEV), _cu([1] * B)
    step_q, step_out = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(B, Hq, D, device=DEV)
    for s in range(steps):
        row = torch.tensor([at[b] + lens[b] + s for b in range(B)], device=DEV)
        q, k, v = (y[row] for y in x)
        E.embla_rope_qkv(shape, cu1, pos, q, k, v, step_q, None, norm_eps=1e-6, k_win=rings[0], v_win=rings[1])
        E.embla_window_decode_ragged(shape, step_q, *rings, pos, step_out)
        assert torch.equal(step_q, turned_q[row])
        R.assert_within(step_out, want[row], tol[row], f"step {s}")
        pos += 1
    _checked()
