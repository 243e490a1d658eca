"""The shared-prefix calls as programs make them, beside test_gpu_shared.py: streams, workspaces,
scores that are not numbers, long stretches of tiles."""
import pytest
import torch

import relu_sparse_kv_gb300 as E
from test_gpu_shared import D, make, run

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
