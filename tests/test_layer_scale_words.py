"""Scales of 8-bit rows are read as whole words where those lie within the tensor.  On the CPU: the functions that
say where words start and which rows leave the tensor, compiled from the kernels' header, for every short row."""
import os
import subprocess

from matrix_state_nonlinear_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include "m2rnn_layer.h"
using namespace m2rnn;
int main() {
  alignas(64) static uint8_t room[8192];
  int words = 0, spared = 0;
  for (int off = 0; off < 4; ++off)
    for (int blocks = 1; blocks <= 37; ++blocks)
      for (long long rows = 1; rows <= 13; ++rows) {
        const uint8_t *from = room + 64 + off, *to = from + rows * blocks;
        for (long long m = 0; m < rows; ++m) {
          const uint8_t* row = from + m * blocks;
          bool leaves = false;
          for (int i = 0; i < blocks; i += 16)
            for (int q = 0; q < 5; ++q) {
              const int at = word_start(row, i) + 4 * q;
              if (at >= blocks) continue;
              const uint8_t* word = row + at;
              if ((reinterpret_cast<uintptr_t>(word) & 3u) || at <= i - 4) return std::printf("not the word of its block\n"), 1;
              leaves = leaves || word < from || word + 4 > to;
              ++words;
            }
          if (leaves && !words_leave(from, rows, blocks, m))
            return std::printf("row %lld of %lld, %d to a row, %d bytes behind a word: out of range\n", m, rows, blocks, off), 1;
          spared += !leaves && words_leave(from, rows, blocks, m);
        }
      }
  // A row that could be read as words and is not costs time alone: those that end with the tensor's last whole word.
  std::printf("%d words, %d rows more than need it\n", words, spared);
  return spared != 0;
}
"""


def test_words_of_scales_lie_within_the_tensor(tmp_path):
    src, exe = tmp_path / "words.cpp", tmp_path / "words"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    include = [f"-I{d}" for d in (build.CSRC, build.INCLUDE, cuda)]
    subprocess.run(["g++", "-std=c++17", *include, str(src), "-o", str(exe)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
