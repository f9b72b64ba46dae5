"""Outputs that share memory with what a call reads are refused, before any GPU
work; slices that lie between each other are not (csrc/layer_overlap.h, compiled
here and compared with a count of bytes)."""
import ctypes
import os
import subprocess

import pytest

from sparse_communication_sharded_gb300 import _scape as C
from sparse_communication_sharded_gb300 import build as B

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_communication_sharded_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include "layer_overlap.h"
using scapek::layer::Span;

static unsigned char mark[4096];
static bool count(int p, int pitch, int width, int rows, int p2, int pitch2, int width2, int rows2) {
  memset(mark, 0, sizeof mark);
  for (int i = 0; i < rows; ++i)
    for (int j = 0; j < width; ++j) mark[p + i * pitch + j] = 1;
  for (int i = 0; i < rows2; ++i)
    for (int j = 0; j < width2; ++j)
      if (mark[p2 + i * pitch2 + j]) return true;
  return false;
}
int main() {
  srand(1);
  long met = 0;
  for (int n = 0; n < 400000; ++n) {
    const int w = rand() % 9, w2 = rand() % 9, rows = rand() % 6, rows2 = rand() % 6;
    int pitch = w + rand() % 12, pitch2 = rand() % 2 ? pitch : w2 + rand() % 12;
    if (pitch2 < w2) pitch2 = w2;
    const int p = 64 + rand() % 90, p2 = 64 + rand() % 90;
    const Span a(mark + p, pitch, w, rows), b(mark + p2, pitch2, w2, rows2);
    const bool want = count(p, pitch, w, rows, p2, pitch2, w2, rows2);
    if (overlap(a, b) != want || overlap(b, a) != want) {
      printf("%d %d %d %d against %d %d %d %d: bytes say %d\n", p, pitch, w, rows, p2, pitch2, w2, rows2, want);
      return 1;
    }
    met += want;
  }
  const Span none(nullptr, 8, 8, 4), all(mark, 8, 8, 4);
  if (overlap(none, all) || !overlap(all, all) || !all.same(Span(mark, 32, 32, 1))) return 2;
  return met > 20000 ? 0 : 3;
}
"""


def test_against_a_count_of_bytes(tmp_path):
    src, exe = tmp_path / "overlap.cpp", tmp_path / "overlap"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


@pytest.fixture(scope="module")
def lib():
    B.build()
    return C.load()


# addresses that no refused call reads, 1 MB apart
PX, PW, PY, PQ, PS, PR, PB, PH, PD, WS = (i << 20 for i in range(1, 11))
BF = C.SCAPE_BF16


def refused(lib, rc):
    assert rc == C.SCAPE_EINVAL
    assert "overlap" in lib.scape_layer_last_error().decode()


@pytest.mark.parametrize("y", [PX, PX + 2, PX - 2, PX + 16 * 128 - 2, PW, PB, PR + 2, PQ, PS])
def test_linear(lib, y):
    refused(lib, lib.scape_layer_linear(PX, 64, PW, 64, PB, PR, 64, 16, 64, 64, 0, y, 64, PQ, 64, PS, None, 0, None))


@pytest.mark.parametrize("dx", [PX, PX + 8, PW, PQ, PS])
def test_linear_input_gradient(lib, dx):
    refused(lib, lib.scape_layer_linear_bwd_input(PX, 64, PW, 64, PQ, 64, PS, 1, 16, 64, 64, dx, 64, None, 0, None))


@pytest.mark.parametrize("dw,db", [(PX, PB), (PQ, PB), (PS, PB), (PH, PX + 64), (PH, PH + 2), (WS, PB)])
def test_linear_weight_gradient(lib, dw, db):
    n = ctypes.c_size_t()
    assert lib.scape_layer_linear_bwd_weight_workspace(PX, 64, None, 0, 16, 64, 64, ctypes.byref(n)) == C.SCAPE_OK
    refused(lib, lib.scape_layer_linear_bwd_weight(PX, 64, None, 0, PQ, 64, PS, 0, 16, 64, 64, dw, 64, db, BF, WS,
                                                   n.value, None))


@pytest.mark.parametrize("y,h", [(PX, PH), (PR, PH), (PW, PH), (PY, PX + 2), (PY, PR - 2), (PY, PW), (PH, PH), (PQ, PH)])
def test_norm(lib, y, h):
    refused(lib, lib.scape_layer_add_rmsnorm(PX, 64, PR, 64, PW, BF, 16, 64, 1e-5, BF, y, 64, h, 64, PB, PQ, 64, PS,
                                             None))


def test_norm_in_the_place_of_an_input_with_another_stride(lib):
    refused(lib, lib.scape_layer_add_rmsnorm(PX, 64, None, 0, PW, BF, 16, 64, 1e-5, BF, PY, 64, PX, 72, PB, None, 0,
                                             None, None))


@pytest.mark.parametrize("dx,dw", [(PH, PB), (PX + 2, PB), (PD + 2, PB), (PR, PB), (PW, PB), (PY, PX), (PY, PY + 8)])
def test_norm_gradient(lib, dx, dw):
    n = ctypes.c_size_t()
    assert lib.scape_layer_add_rmsnorm_bwd_workspace(16, 64, ctypes.byref(n)) == C.SCAPE_OK
    refused(lib, lib.scape_layer_add_rmsnorm_bwd(PX, 64, PH, 64, PW, BF, PR, PD, 64, 16, 64, BF, dx, 64, dw, BF, WS,
                                                 n.value, None))


def test_pack_unpack_and_activation_gradient(lib):
    refused(lib, lib.scape_layer_pack8(PX, 64, BF, 16, 64, PX, 64, PS, None))
    refused(lib, lib.scape_layer_pack8(PX, 64, BF, 16, 64, PQ, 64, PX + 100, None))
    refused(lib, lib.scape_layer_pack8(PX, 64, BF, 16, 64, PQ, 64, PQ, None))
    refused(lib, lib.scape_layer_unpack8(PQ, 64, PS, 16, 64, 0, PQ, 64, BF, None))
    refused(lib, lib.scape_layer_unpack8(PQ, 64, PS, 16, 64, 0, PS, 64, BF, None))
    refused(lib, lib.scape_layer_act_grad(PX, 64, PQ, 64, PS, 16, 64, 1, PX + 2, 64, BF, None))
    refused(lib, lib.scape_layer_act_grad(PX, 64, PQ, 64, PS, 16, 64, 1, PX, 128, BF, None))
    refused(lib, lib.scape_layer_act_grad(PX, 64, PQ, 64, PS, 16, 64, 1, PQ, 64, BF, None))
