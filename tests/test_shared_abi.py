"""CPU-side checks of the cache-row and shared-prefix calls: what they refuse before touching the
device, what is a no-op, and the work split of the shared-prefix decode (compiled from its
header with g++)."""
import ctypes
import os
import subprocess

import pytest
import torch

import relu_sparse_kv_gb300 as E
from relu_sparse_kv_gb300 import build as B

OK, INVALID, UNSUPPORTED = 0, 1, 2
A = [ctypes.c_void_p(256 * (k + 1)) for k in range(16)]  # aligned, never dereferenced
ODD = ctypes.c_void_p(264)                               # 8-byte aligned only


@pytest.fixture(scope="module")
def lib():
    B.build()
    return E.library()


def _shape(**kw):
    d = dict(batch=2, n_q_heads=16, n_kv_heads=4, head_dim=128, ctx_len=100, cache_stride=128)
    d.update(kw)
    return ctypes.byref(E._Shape(**d))


def test_quantize_refusals(lib):
    f = lib.embla_quantize_kv_e4m3
    ptrs = A[:6]
    assert f(None, 0, 1, *ptrs, None) == INVALID
    assert f(_shape(head_dim=64), 0, 1, *ptrs, None) == UNSUPPORTED
    assert f(_shape(n_q_heads=12), 0, 1, *ptrs, None) == UNSUPPORTED  # G = 3
    assert f(_shape(n_kv_heads=3), 0, 1, *ptrs, None) == INVALID
    for pos, n in ((-1, 1), (0, -1), (128, 1), (0, 129), (100, 29), (2 ** 62, 2 ** 62)):
        assert f(_shape(), pos, n, *ptrs, None) == INVALID, (pos, n)
    for k in range(6):
        assert f(_shape(), 0, 1, *ptrs[:k], None, *ptrs[k + 1:], None) == INVALID
        assert f(_shape(), 0, 1, *ptrs[:k], ODD, *ptrs[k + 1:], None) == INVALID
    big = _shape(batch=1 << 20, cache_stride=1 << 30)
    assert f(big, 0, 1 << 29, *ptrs, None) == UNSUPPORTED  # 2^51 rows
    assert f(_shape(batch=0), 0, 1, *[None] * 6, None) == OK
    assert f(_shape(), 5, 0, *[None] * 6, None) == OK


def test_dequantize_refusals(lib):
    f = lib.embla_dequantize_kv_e4m3
    ptrs = A[:6]
    assert f(None, 0, 1, *ptrs, 1, None) == INVALID
    assert f(_shape(head_dim=256), 0, 1, *ptrs, 1, None) == UNSUPPORTED
    for pos, n, stride in ((-1, 1, 1), (0, -1, 1), (128, 1, 1), (0, 129, 200), (0, 5, 4), (0, 0, -1)):
        assert f(_shape(), pos, n, *ptrs, stride, None) == INVALID, (pos, n, stride)
    for k in range(6):
        assert f(_shape(), 0, 1, *ptrs[:k], None, *ptrs[k + 1:], 1, None) == INVALID
        assert f(_shape(), 0, 1, *ptrs[:k], ODD, *ptrs[k + 1:], 1, None) == INVALID
    assert f(_shape(batch=0), 0, 1, *[None] * 6, 1, None) == OK
    assert f(_shape(), 128, 0, *[None] * 6, 0, None) == OK


def _full(lib, shape=None, plen=300, pstride=300, q=A[0], kp=A[1], vp=A[2], k=A[3], v=A[4], alpha=1.0,
          c=1.0, eps=1e-6, out=A[5], ns=A[6], sel=A[7], sstride=400, hist=A[8], ws=A[9], wsb=1 << 40):
    return lib.embla_full_decode_shared(shape or _shape(), plen, pstride, q, kp, vp, k, v, alpha, c, eps, out,
                                        ns, sel, sstride, hist, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(plen=-1), INVALID),
    (dict(pstride=299), INVALID),
    (dict(plen=2 ** 31 - 357, pstride=2 ** 31), INVALID),   # 2^31 - 257 keys of context in all
    (dict(plen=2 ** 62, pstride=2 ** 62), INVALID),
    (dict(alpha=0.0), INVALID), (dict(alpha=float("nan")), INVALID), (dict(c=-1.0), INVALID),
    (dict(eps=float("inf")), INVALID),
    (dict(q=None), INVALID), (dict(kp=None), INVALID), (dict(vp=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(out=None), INVALID), (dict(ns=None), INVALID), (dict(ws=None), INVALID),
    (dict(sel=None), INVALID), (dict(hist=None), INVALID),  # both or neither
    (dict(sstride=399), INVALID),
    (dict(q=ODD), INVALID), (dict(kp=ODD), INVALID), (dict(vp=ODD), INVALID), (dict(k=ODD), INVALID),
    (dict(v=ODD), INVALID), (dict(out=ODD), INVALID), (dict(ns=ODD), INVALID), (dict(sel=ODD), INVALID),
    (dict(hist=ODD), INVALID), (dict(ws=ODD), INVALID),
    (dict(shape=_shape(head_dim=64)), UNSUPPORTED), (dict(shape=_shape(n_q_heads=12)), UNSUPPORTED),
    (dict(shape=_shape(ctx_len=129)), INVALID), (dict(shape=_shape(batch=-1)), INVALID),
    (dict(shape=_shape(batch=1 << 27)), UNSUPPORTED),       # 2^31 query heads
    (dict(pstride=1 << 32), UNSUPPORTED), (dict(shape=_shape(cache_stride=1 << 32)), UNSUPPORTED),  # 1 TB per plane
])
def test_full_shared_refusals(lib, kw, status):
    assert _full(lib, **kw) == status


def test_full_shared_empty_batch_is_a_no_op(lib):
    assert _full(lib, shape=_shape(batch=0), q=None, kp=None, vp=None, k=None, v=None, out=None, ns=None,
                 sel=None, hist=None, ws=None, wsb=0) == OK


def _sparse(lib, shape=None, plen=300, pstride=300, q=A[0], kp=A[1], vp=A[2], k=A[3], v=A[4], idx=A[5],
            istride=1152, count=A[6], tau=0.1, out=A[7]):
    return lib.embla_sparse_decode_shared(shape or _shape(), plen, pstride, q, kp, vp, k, v, idx, istride, count,
                                          tau, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(plen=-1), INVALID), (dict(pstride=299), INVALID), (dict(istride=-1), INVALID),
    (dict(tau=float("inf")), INVALID),
    (dict(q=None), INVALID), (dict(kp=None), INVALID), (dict(vp=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(idx=None), INVALID), (dict(count=None), INVALID), (dict(out=None), INVALID),
    (dict(q=ODD), INVALID), (dict(kp=ODD), INVALID), (dict(vp=ODD), INVALID), (dict(k=ODD), INVALID),
    (dict(v=ODD), INVALID), (dict(idx=ODD), INVALID), (dict(count=ODD), INVALID), (dict(out=ODD), INVALID),
    (dict(shape=_shape(head_dim=64)), UNSUPPORTED), (dict(shape=_shape(ctx_len=-1)), INVALID),
    (dict(shape=_shape(batch=1 << 27)), UNSUPPORTED),
])
def test_sparse_shared_refusals(lib, kw, status):
    assert _sparse(lib, **kw) == status


def test_sparse_shared_empty_batch_is_a_no_op(lib):
    assert _sparse(lib, shape=_shape(batch=0), q=None, kp=None, vp=None, k=None, v=None, idx=None, count=None,
                   out=None) == OK


def test_binding_refuses_host_tensors_and_wrong_types():
    sh = E.Shape(1, 16, 4, 128, 2, 4)
    rows = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16)
    codes, scales = torch.zeros(1, 4, 4, 128, dtype=torch.uint8), torch.ones(1, 4, 4)
    with pytest.raises(ValueError):
        E.embla_quantize_kv_e4m3(sh, 0, rows, rows, codes, scales, codes, scales)
    with pytest.raises(TypeError):
        E.embla_quantize_kv_e4m3(sh, 0, rows.float(), rows, codes, scales, codes, scales)
    with pytest.raises(ValueError):
        E.embla_dequantize_kv_e4m3(sh, 0, codes, scales, codes, scales, rows, rows)
    q, pre = torch.zeros(1, 16, 128, dtype=torch.bfloat16), torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        E.embla_full_decode_shared(sh, 8, q, pre, pre, rows, rows, torch.zeros(1, 16, 128),
                                   torch.zeros(1, 4, dtype=torch.int32))
    idx, count = torch.zeros(1, 4, 8, dtype=torch.int32), torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        E.embla_sparse_decode_shared(sh, 8, q, pre, pre, rows, rows, idx, count, torch.zeros(1, 16, 128))


HARNESS = r"""
#include <cstdio>
#include <vector>
#include "shared_prefix.h"
using namespace embla;
// Every tile of every row block belongs to exactly one stretch; a stretch's record slot is its
// own and lies inside the workspace; the records of a row are those of the stretches that hold
// prefix tiles of its KV head or own tiles of its sequence.
int main() {
  const int Bs[] = {1, 2, 15, 16, 17, 32, 33, 64, 65, 97, 160};
  const long Ps[] = {0, 1, 127, 128, 129, 700, 2048, 33000};
  const long ns[] = {0, 1, 128, 129, 400, 3000};
  const int smss[] = {1, 2, 5, 20, 152};
  for (int G : {4, 8})
    for (int Hkv : {1, 2, 4})
      for (int B : Bs)
        for (long P : Ps)
          for (long n : ns)
            for (int sms : smss) {
              const SharedSplit sp = shared_split(B, Hkv, G, P, n, sms);
              if (P + n == 0) {
                if (sp.ctas() != 0 || shared_workspace_bytes(sp) != 0) return 1;
                continue;
              }
              if (sp.ctas() < sp.blocks || (sp.ctas() > sms && sp.ctas() > sp.blocks)) return 2;
              if (!sp.fits()) return 12;
              const long slots = sp.slot(sp.blocks, 0, 0);
              std::vector<char> used(slots, 0);
              std::vector<long> cta_of;  // (row block, piece) by CTA
              int seqs_seen = 0;
              for (int rb = 0; rb < sp.blocks; ++rb) {
                const long gt = sp.group_tiles(rb), T = gt * Hkv, Q = sp.pieces(rb);
                if (Q < 1 || Q > T) return 3;
                seqs_seen += sp.sequences(rb);
                long covered = 0;
                for (long q = 0; q < Q; ++q) {
                  const long cta = (long)rb * sp.ctas_full + q;
                  if (cta >= sp.ctas() || sp.block_of_cta(cta) != rb) return 4;
                  const long b = sp.piece_start(q, T, Q), e = sp.piece_start(q + 1, T, Q);
                  if (b != covered || e <= b) return 5;
                  covered = e;
                  for (long g = b / gt; g <= (e - 1) / gt; ++g) {
                    const long s = sp.slot(rb, q, g);
                    if (s < 0 || s >= slots || used[s]) return 6;
                    used[s] = 1;
                  }
                  if (sp.piece_of_tile(b, T, Q) != q || sp.piece_of_tile(e - 1, T, Q) != q) return 7;
                }
                if (covered != T) return 8;
              }
              if (seqs_seen != B) return 9;
            }
  // the CTAs of the row blocks walk the same prefix tiles at the same time
  const SharedSplit two = shared_split(64, 4, 4, 65536, 1024, 152);
  if (two.blocks != 2 || two.ctas_full != 76 || two.ctas_last != 76) return 10;
  if (shared_split(32, 4, 4, 32768, 300, 152).ctas() != 152) return 11;
  std::puts("ok");
  return 0;
}
"""


def test_shared_work_split_host_logic(lib, tmp_path):
    src, exe = tmp_path / "shared.cpp", tmp_path / "shared"
    src.write_text(HARNESS)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-I" + B.CSRC, "-I/usr/local/cuda/include", str(src),
                        os.path.join(B.BUILD, "shared_decode.o"), "-o", str(exe), "-L/usr/local/cuda/lib64",
                        "-lcudart_static", "-ldl", "-lpthread", "-lrt"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stdout)
