"""What the binding of the shared-prefix calls takes and refuses (no GPU: the library is a
stand-in): a side without keys needs no tensors, as the C calls have it."""
import pytest
import torch

import relu_sparse_kv_gb300 as E
from test_binding_workspaces import B, D, HKV, HQ, Library, bf16, f32, i32

Q, OUT, COUNT, IDX = bf16(B, HQ, D), f32(B, HQ, D), i32(B, HKV), i32(B, HKV, 8)
PREFIX = bf16(HKV, 5, D), bf16(HKV, 5, D)
OWN = bf16(B, HKV, 7, D), bf16(B, HKV, 7, D)
NONE = (None, None)


def full(shape, prefix_len, prefix, own):
    E.embla_full_decode_shared(shape, prefix_len, Q, *prefix, *own, OUT, COUNT)


def sparse(shape, prefix_len, prefix, own):
    E.embla_sparse_decode_shared(shape, prefix_len, Q, *prefix, *own, IDX, COUNT, OUT)


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(E, "library", lambda: lib)
    monkeypatch.setattr(E, "_stream", lambda *a: None)

    def check_here(*tensors):  # the checks, but for the device
        for t, dtype, shape, name in tensors:
            if t is None or t.dtype is not dtype or tuple(t.shape) != tuple(shape):
                raise ValueError(name)
        return 0

    monkeypatch.setattr(E, "_check_here", check_here)
    return lib


@pytest.mark.parametrize("call", [full, sparse])
@pytest.mark.parametrize("prefix_len,n,prefix,own,planes", [
    (4, 6, PREFIX, OWN, (5, *PREFIX, *OWN)), (0, 6, NONE, OWN, (0, *NONE, *OWN)),
    (0, 6, PREFIX, OWN, (5, *PREFIX, *OWN)), (4, 0, PREFIX, NONE, (5, *PREFIX, *NONE)),
    (0, 0, NONE, NONE, (0, *NONE, *NONE)),
])
def test_sides_without_keys_may_be_none(lib, call, prefix_len, n, prefix, own, planes):
    call(E.Shape(B, HQ, HKV, D, n, 7), prefix_len, prefix, own)
    (_, args), = lib.calls
    stride, *tensors = planes
    assert args[1:3] == (prefix_len, stride)
    assert args[4:8] == tuple(None if t is None else t.data_ptr() for t in tensors)


@pytest.mark.parametrize("call", [full, sparse])
@pytest.mark.parametrize("prefix_len,n,prefix,own", [
    (4, 6, NONE, OWN), (6, 6, PREFIX, OWN), (4, 6, (PREFIX[0], None), OWN), (0, 6, (None, PREFIX[1]), OWN),
    (0, 6, (PREFIX[0], None), OWN), (4, 6, PREFIX, NONE), (4, 0, PREFIX, (OWN[0], None)),
    (4, 0, PREFIX, (None, OWN[1])), (-1, 6, NONE, OWN), (4, 6, (PREFIX[0][0], PREFIX[1]), OWN),
])
def test_sides_with_keys_and_half_sides_are_refused(lib, call, prefix_len, n, prefix, own):
    with pytest.raises(ValueError):
        call(E.Shape(B, HQ, HKV, D, n, 7), prefix_len, prefix, own)
    assert lib.calls == []
