"""Which records the finishing kernel of the shared-prefix decode adds up for a row: host logic, compiled
from its header with g++ and compared with the pieces that hold tiles of the row."""
import os
import subprocess

from relu_sparse_kv_gb300 import build as B

HARNESS = r"""
#include <cstdio>
#include <vector>
#include "shared_prefix.h"
using namespace embla;
int main() {
  long rows = 0;
  for (int G : {4, 8})
    for (int Hkv : {1, 2, 4})
      for (int B : {1, 2, 15, 16, 17, 33, 64, 97, 160})
        for (long P : {0L, 1L, 128L, 129L, 700L, 2048L, 33000L})
          for (long n : {0L, 1L, 128L, 129L, 400L, 3000L})
            for (int sms : {1, 2, 5, 20, 152}) {
              const SharedSplit sp = shared_split(B, Hkv, G, P, n, sms);
              if (P + n == 0) continue;
              for (int rb = 0; rb < sp.blocks; ++rb) {
                const long gt = sp.group_tiles(rb), T = gt * Hkv, Q = sp.pieces(rb);
                // piece of each tile of the row block's list
                std::vector<int> piece(T);
                for (long q = 0; q < Q; ++q)
                  for (long t = sp.piece_start(q, T, Q); t < (long)sp.piece_start(q + 1, T, Q); ++t) piece[t] = q;
                for (int g = 0; g < Hkv; ++g)
                  for (int seq = 0; seq < sp.sequences(rb); ++seq, ++rows) {
                    std::vector<int> want;
                    auto hold = [&](long t) {
                      if (want.empty() || want.back() != piece[t]) want.push_back(piece[t]);
                    };
                    for (long t = 0; t < sp.tp; ++t) hold(g * gt + t);
                    for (long t = 0; t < sp.ts; ++t) hold(g * gt + sp.tp + seq * sp.ts + t);
                    const SharedSplit::RowPieces r = sp.row_pieces(rb, seq, g);
                    std::vector<int> got;
                    for (int k = 0; k < r.prefix; ++k) got.push_back(r.first + k);
                    for (int k = 0; k < r.rest; ++k) got.push_back(r.own + k);
                    if (got != want) return 1;
                  }
              }
            }
  std::printf("ok %d\n", rows > 1000000);
  return 0;
}
"""


def test_a_rows_records_are_those_of_the_pieces_with_its_tiles(tmp_path):
    B.build()
    src, exe = tmp_path / "records.cpp", tmp_path / "records"
    src.write_text(HARNESS)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-I" + B.CSRC, "-I/usr/local/cuda/include", str(src),
                        os.path.join(B.BUILD, "shared_decode.o"), "-o", str(exe), "-L/usr/local/cuda/lib64",
                        "-lcudart_static", "-ldl", "-lpthread", "-lrt"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok 1", (r.returncode, r.stdout)
