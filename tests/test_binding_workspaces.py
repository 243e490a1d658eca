"""Workspaces that the binding makes for a call (no GPU: the library and the allocator are stand-ins):
allocated with the call's stream current, so the caching allocator orders their reuse by it."""
import contextlib

import pytest
import torch

import relu_sparse_kv_gb300 as E

B, HQ, HKV, D, N = 1, 8, 2, 128, 4
SHAPE = E.Shape(B, HQ, HKV, D, N, N)


class Library:
    """Every size is 64, every call succeeds and its arguments are kept."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            if name.endswith("_workspace_size"):
                return 64
            self.calls.append((name, args))
            return 0
        return fn


class Stream:
    cuda_stream = 0x5EED


def f32(*s):
    return torch.zeros(*s)


def bf16(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def u8(*s):
    return torch.zeros(*s, dtype=torch.uint8)


Q, CACHE, OUT = bf16(B, HQ, D), bf16(B, HKV, N, D), f32(B, HQ, D)
CODES, SCALES = u8(B, HKV, N, D), f32(B, HKV, N)
COUNT, SCORES, HIST, IDX = i32(B, HKV), f32(B, HKV, N), i32(B, HKV, E.HIST_BINS), i32(B, HKV, 1152)
PER_HEAD = f32(B, HQ, N), i32(B, HQ, E.HIST_BINS), i32(B, HQ, 1152), i32(B, HQ)
PREFIX = bf16(HKV, 3, D)
CODED = CODES, SCALES, CODES, SCALES
CALLS = {
    "embla_full_decode": (SHAPE, Q, CACHE, CACHE, OUT, COUNT),
    "embla_full_decode_e4m3": (SHAPE, Q, *CODED, OUT, COUNT),
    "embla_full_decode_select": (SHAPE, Q, CACHE, CACHE, OUT, COUNT, SCORES, HIST, IDX, COUNT),
    "embla_full_decode_e4m3_select": (SHAPE, Q, *CODED, OUT, COUNT, SCORES, HIST, IDX, COUNT),
    "embla_full_decode_head_scores": (SHAPE, Q, CACHE, CACHE, OUT, COUNT, *PER_HEAD[:2]),
    "embla_full_decode_shared": (SHAPE, 3, Q, PREFIX, PREFIX, CACHE, CACHE, OUT, COUNT),
    "embla_select_topk": (SHAPE, SCORES, HIST, IDX, COUNT),
    "embla_select_topk_per_head": (SHAPE, *PER_HEAD),
    "embla_sparse_decode": (SHAPE, Q, CACHE, CACHE, IDX, COUNT, OUT),
    "embla_sparse_decode_e4m3": (SHAPE, Q, *CODED, IDX, COUNT, OUT),
    "embla_sparse_decode_per_head": (SHAPE, Q, CACHE, CACHE, *PER_HEAD[2:], OUT),
    "embla_prefill": (SHAPE, bf16(B, HQ, N, D), CACHE, CACHE, f32(B, HQ, N, D)),
    "embla_relu2_mlp": (bf16(512), bf16(8, 512), bf16(8, 512), f32(512), i32(1)),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_call_makes_its_workspace_on_its_own_stream(name, monkeypatch):
    lib, current, made = Library(), [None], []
    monkeypatch.setattr(E, "library", lambda: lib)
    monkeypatch.setattr(E, "_check", lambda *a, **k: None)
    monkeypatch.setattr(E, "_check_here", lambda *a: 0)

    @contextlib.contextmanager
    def stream_context(s):
        current.append(s)
        yield
        current.pop()

    empty = torch.empty

    def allocate(*args, **kw):
        t = empty(*args, **kw)
        made.append((t.data_ptr(), current[-1]))
        return t

    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(torch, "empty", allocate)
    stream = Stream()
    getattr(E, name)(*CALLS[name], stream=stream)
    (called, args), = lib.calls
    assert called == name and args[-1] == stream.cuda_stream
    (pointer, owner), = made
    assert pointer in args and owner is stream
    assert current == [None]
