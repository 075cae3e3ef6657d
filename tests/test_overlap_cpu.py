"""Where tensors of rows share memory (csrc/host_util.h), on the host against a count of every byte, and the entry
points that refuse it (nothing is launched)."""

import os
import shutil
import subprocess

import pytest

import paged_decode_attention_fp8_gb300 as fm
from tests.test_operators_capi_cpu import P, _append, _apply, _decode, _read

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_decode_attention_fp8_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <map>
#include <random>
#include "host_util.h"
using namespace fp8mla;

static std::map<int64_t, int> bytes(const Rows& r) {  // how many rows hold each byte
  std::map<int64_t, int> m;
  for (int64_t i = 0; i < r.n; ++i)
    for (int64_t h = 0; h < r.heads; ++h)
      for (int64_t x = 0; x < r.width; ++x) ++m[r.at + i * r.token + h * r.head + x];
  return m;
}

int main() {
  std::mt19937 g(1);
  auto pick = [&](int lo, int hi) { return static_cast<int64_t>(lo + g() % (hi - lo + 1)); };
  int shared = 0, apart = 0, own = 0, sound = 0, exact = 0;
  for (int t = 0; t < 60000; ++t) {
    Rows a{1000 + pick(0, 40), pick(-24, 24), pick(-24, 24), pick(1, 6), pick(1, 5), pick(1, 9)};
    Rows b = a;
    b.at = 1000 + pick(0, 90);
    b.n = pick(1, 6), b.heads = pick(1, 5);
    if (t % 3 == 0) b.width = pick(1, 9);
    const bool same = t % 5 != 0;
    if (!same) b.token = pick(-24, 24), b.head = pick(-24, 24);
    const auto ma = bytes(a), mb = bytes(b);
    bool hit = false, twice = false;
    for (const auto& x : ma) hit |= mb.count(x.first) > 0, twice |= x.second > 1;
    const bool said = rows_overlap(a, b);
    if (hit && !said) return 1;  // never missed
    if (same && said != hit) return 2;
    if (rows_overlap(b, a) != said) return 3;
    if (rows_overlap_themselves(a) != twice) return 4;
    if (rows_overlap(a, Rows{b.at, 0, 0, 1, 1, b.width}) != [&] {
          for (int64_t x = 0; x < b.width; ++x) if (ma.count(b.at + x)) return true;
          return false; }()) return 5;  // a block against rows: exact
    (hit ? shared : apart)++, (twice ? own : sound)++, exact += said == hit;
  }
  if (shared < 5000 || apart < 5000 || own < 5000 || sound < 5000 || exact < 55000) return 6;
  const Rows none{1000, 8, 8, 0, 4, 8}, far{1000, INT64_MAX, 8, 3, 4, 8}, one{1000, 8, 8, 1, 1, 8};
  if (rows_overlap(none, one) || rows_overlap_themselves(none)) return 7;
  if (!rows_overlap(far, one) || !rows_overlap_themselves(far)) return 8;
  if (!rows_overlap_themselves(rows_of(&none, INT64_MAX / 2, 1, 2, 1, 8, 4))) return 9;
  if (clobbers(one, one) || !clobbers(one, Rows{1004, 8, 8, 1, 1, 8}) || block_of(nullptr, 8).heads != 0) return 10;
  // a projection's output split into heads, 2^20 tokens: queries, keys and values interleave
  const Rows q = rows_of(&none, 48 * 128, 128, 1 << 20, 32, 128, 2);
  Rows k = q;
  k.at += 32 * 256, k.heads = 8;
  if (rows_overlap(q, k) || rows_overlap_themselves(q)) return 11;
  k.at -= 2;
  if (!rows_overlap(q, k)) return 12;
  std::puts("overlap ok");
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_shared_bytes(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "overlap ok", r.returncode


APART = dict(qo=2 * P, ko=3 * P, k=4 * P)
SPLIT = dict(qs=(48 * 128, 128), qos=(48 * 128, 128), ks=(48 * 128, 128), kos=(48 * 128, 128), k=P + 32 * 256)


@pytest.mark.parametrize("over", [
    dict(APART, qos=(4096, 64)),                         # neighbouring heads share half of theirs
    dict(APART, qos=(100, 100)),
    dict(APART, qos=(128, 128)),                         # token 1's head 0 is token 0's head 1
    dict(APART, kos=(1000, 128)),
    dict(APART, ko=2 * P + 256),                         # the outputs one over the other
    dict(APART, qo=P + 16), dict(APART, qo=P, qos=(8192, 128)),  # over the input, not in its place
    dict(APART, ko=P), dict(APART, qo=4 * P),            # over the other's input
    dict(SPLIT, ko=P + 31 * 256), dict(SPLIT, qo=P + 256, ko=P + 40 * 256)])
def test_rotation_refuses_shared_memory(over):
    assert _apply(**over) == 1


OK_APPEND = dict(v=2 * P, kc=3 * P, vc=4 * P, k_blk=5 * P, v_blk=6 * P, q=7 * P, qo=8 * P)


@pytest.mark.parametrize("over", [dict(vc=3 * P), dict(vc=3 * P + 64 * 8 * 16 * 64 - 16), dict(v_blk=5 * P + 16),
                                  dict(k_blk=3 * P + 16), dict(qo=3 * P), dict(qo=P + 16), dict(qo=2 * P + 32),
                                  dict(qo=7 * P + 16), dict(k=3 * P + 32), dict(v=3 * P), dict(q=4 * P),
                                  dict(qs=(5120, 128), qo=7 * P)])
def test_append_refuses_shared_memory(over):
    assert _append(**{**OK_APPEND, **over}) == 1


def test_append_refuses_shared_row_scales():
    rows = dict(OK_APPEND, dtype=fm.KV_E4M3, k_scale=None, v_scale=None, k_blk=None, v_blk=None, k_rows=9 * P)
    assert _append(**rows, v_rows=9 * P + 4) == 1
    assert _append(**rows, v_rows=4 * P) == 1


@pytest.mark.parametrize("over", [dict(), dict(out=P + 64 * 8 * 16 * 64 - 16), dict(out=3 * P, blk=3 * P + 16)])
def test_read_refuses_to_write_over_the_cache(over):
    assert _read(**over) == 1


@pytest.mark.parametrize("over", [dict(lse=P), dict(out=P + 16), dict(lse=2 * P, out=2 * P - 16),
                                  dict(lse=3 * P, ws=3 * P, splits=2, mb=64, out=2 * P),
                                  dict(out=3 * P, ws=3 * P + 256, splits=2, mb=64, lse=2 * P),
                                  dict(ws=P, out=2 * P, lse=3 * P, splits=2, mb=64)])
def test_attention_refuses_shared_outputs(over):
    assert _decode(**over) == 1
