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
