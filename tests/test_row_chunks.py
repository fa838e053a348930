"""Chunks of rows in the backward of the norms between blocks: the plan and the rows of each chunk (csrc/row_chunks.h,
which the kernels use), compiled by the host compiler. No GPU is needed."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "swiglu_ffn_backward_gb300", "csrc")

# M, rows of a gate row, groups that take chunks, distance of a chunk's rows: small sizes all, and those of calls
PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "row_chunks.h"
using namespace swg;
template <bool kApart, typename Int>
static void check(const BnChunks& k, int64_t M, int64_t per_gate, const char* what) {
  std::vector<char> seen(M, 0);
  const bool shared = k.segment == per_gate;  // rows share a gate row (or there is none): the chunk's is its segment
  int64_t empty = 0, bad_row = 0, bad_gate = 0, twice = 0, longest = 0, gates = M / k.segment;
  for (int64_t c = 0; c < k.chunks; ++c) {
    const ChunkRows<Int> w = chunk_rows<kApart, Int>(k, static_cast<Int>(c));
    const int64_t apart = kApart ? k.apart : 1, gate = c / k.per_segment;
    bad_gate += static_cast<int64_t>(w.segment) != gate || gate >= gates;  // the row of the gate that is read, rows or none
    int64_t n = 0;
    for (int64_t r = w.first; r < static_cast<int64_t>(w.end); r += apart, ++n) {
      if (r >= M) { ++bad_row; continue; }
      bad_gate += shared && r / per_gate != gate;
      twice += seen[r]++;
    }
    empty += n == 0;
    if (n > longest) longest = n;
  }
  int64_t missing = 0;
  for (char s : seen) missing += s == 0;
  std::printf("%s %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld\n", what, (long long)M, (long long)per_gate,
              (long long)k.apart, (long long)k.chunks, (long long)empty, (long long)bad_row, (long long)bad_gate,
              (long long)twice, (long long)missing, (long long)longest, (long long)(M / k.segment));
}
static void all(int64_t M, int64_t per_gate, int64_t units, int64_t apart) {
  const BnChunks k = chunks_of(M, per_gate, units, apart);
  check<true, int64_t>(k, M, per_gate, "registers");
  check<true, uint32_t>(k, M, per_gate, "ring");
  if (apart == 1) check<false, uint32_t>(k, M, per_gate, "whole");
}
int main() {
  for (int64_t M = 1; M <= 70; ++M)
    for (int64_t per_gate = 1; per_gate <= M; ++per_gate)
      for (int64_t apart = 1; apart <= 8; apart *= 2)
        if (M % per_gate == 0)
          for (int64_t units : {1, 7, 304}) all(M, per_gate, units, apart);
  const int64_t sizes[][2] = {{60001, 60001}, {40000, 2}, {33000, 3}, {20011, 20011}, {60000, 20000}, {2003, 2003},
                              {100000, 5}, {99999, 9}, {16384, 2048}, {220000, 220000}, {9999, 7 * 1}, {65536, 64}};
  for (const auto& s : sizes)
    for (int64_t apart = 1; apart <= 8; apart *= 2)
      for (int64_t units : {38, 152, 304, 2432})
        if (s[0] % s[1] == 0) all(s[0], s[1], units, apart);
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("chunks")
    (d / "chunks.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O2", "-I", CSRC, str(d / "chunks.cpp"), "-o", str(d / "chunks")], check=True)
    out = subprocess.run([str(d / "chunks")], check=True, capture_output=True, text=True).stdout
    names = ("kernel", "M", "per_gate", "apart", "chunks", "empty", "bad_row", "bad_gate", "twice", "missing", "longest",
             "segments")
    return [dict(zip(names, [v if i == 0 else int(v) for i, v in enumerate(line.split())])) for line in out.splitlines()]


def test_every_row_once(plans):
    assert len(plans) > 3000
    for p in plans:
        assert p["bad_row"] == p["twice"] == p["missing"] == 0, p
        assert p["longest"] <= 128, p


def test_a_chunks_gate_row_is_there(plans):
    # of chunks without rows too, whose first row is none of their segment
    assert any(p["empty"] > 0 for p in plans)
    for p in plans:
        assert p["bad_gate"] == 0, p


def test_no_more_chunks_than_rows(plans):
    # a chunk's column sums are two fp32 rows of the workspace
    for p in plans:
        # a segment's runs of rows `apart` from one another differ by one row, and are cut alike
        assert p["chunks"] <= p["M"] + (p["apart"] - 1) * p["segments"], p
        if p["per_gate"] < p["apart"] and p["per_gate"] > 1:
            assert p["chunks"] == p["M"] and p["empty"] == 0, p


def test_workspace_of_short_runs():
    # ragged rows whose gate rows serve two or three each: below four 16-bit tensors and a bit
    from swiglu_ffn_backward_gb300 import _binding as b
    for M, N, G in ((40000, 1001, 20000), (21000, 1001, 7000), (33000, 515, 16500), (9000, 4003, 1800)):
        assert b.lib.block_norm_bwd_workspace_size(M, N, G) <= M * (8 * N + 4) + 16
