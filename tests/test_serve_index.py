"""The index arithmetic that the single-token serving kernels share with the
host (csrc/serve_index.h), in a host program against plain counting, with signed
overflow trapped."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "kv_cache_attention_flash_b200", "csrc")


def host(tmp_path, body):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text('#include <cstdint>\n#include <cstdio>\n#include <initializer_list>\n#include "serve_index.h"\nusing namespace fdllm;\n'
                   '#define CHECK(x, ...) do { if (!(x)) { printf(__VA_ARGS__); return 1; } } while (0)\n'
                   "int main() {\n" + body + "\n  return 0;\n}\n")
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], stdout=subprocess.PIPE, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


def test_the_last_pass_of_every_stage_of_a_ring(tmp_path):
    """A ring of 1 to 6 stages is filled stage by stage and left after any number
    of tiles. A wait for a stage's copies must return only when they are there: a
    barrier that has completed c phases lets a wait for parity p through when
    (c & 1) != p. Also at the point where it has already completed them."""
    host(tmp_path, """
  for (int stages = 1; stages <= 6; ++stages)
    for (int tiles = 0; tiles <= 40; ++tiles) {
      int fills[6] = {0};                 // of each stage so far
      int next = 0, round = 0;
      for (int t = 0; t < tiles; ++t) {
        ++fills[next];
        if (++next == stages) next = 0, ++round;
      }
      for (int s = 0; s < stages; ++s) {
        const int pass = last_pass(s, next, round);
        CHECK(pass == fills[s] - 1, "%d stages, %d tiles, stage %d: pass %d", stages, tiles, s, pass);
        if (pass < 0) continue;
        const int parity = pass & 1, under_way = fills[s] - 1, there = fills[s];
        CHECK((under_way & 1) == parity, "the wait would return before the copies are there");
        CHECK((there & 1) != parity, "the wait would not return");
      }
    }""")


def test_the_tiles_of_a_range_of_slots(tmp_path):
    """Against counting, and at lengths whose rounding up leaves 31 bits."""
    host(tmp_path, """
  for (int tile : {32, 64})
    for (int first = 0; first <= 200; ++first)
      for (int len = first; len <= 400; ++len) {
        int seen = 0;
        for (int t = 0; t * tile < 400; ++t) {
          bool any = false;
          for (int s = t * tile; s < (t + 1) * tile; ++s) any = any || (s >= first && s < len);
          seen += any;
        }
        CHECK(tiles_of(first, len, tile) == (len > first ? seen : 1), "%d %d %d", first, len, tile);
      }
  const int most = 2147483646;
  for (int tile : {32, 64})
    for (int cut = 0; cut < 200; ++cut) {
      const long long want = ((long long)most - cut + tile - 1) / tile;
      CHECK(tiles_of(0, most - cut, tile) == want, "%d: %d", cut, tiles_of(0, most - cut, tile));
    }""")
