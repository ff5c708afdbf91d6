"""How CTAs share the items of decay attention's pass (csrc/decay_share.h), gone through on
the host for GPUs of every size: each chunk of each item is some CTA's, no CTA has more
parts than its table has places, and what two CTAs share is begun by the first of them
before all else and ended by the next after all else."""
import ctypes
import os
import shutil
import subprocess

import pytest

from weight_rnn_gb300 import build as wbuild

SOURCE = r"""
#include <vector>
#include "decay_share.h"
using namespace delta::decay;
extern "C" int table() { return kParts; }
extern "C" int shares(long long items, int passes, long long sms) { return share_items(items, passes, sms); }
extern "C" int parts(unsigned items, unsigned chunks, unsigned cta, unsigned ctas) {
  Run r = {};
  int k = 0;
  while (shared_part(items, chunks, cta, ctas, k, r)) ++k;
  return k;
}
// 0, or what is wrong
extern "C" int wrong(unsigned items, unsigned chunks, unsigned ctas) {
  std::vector<unsigned> next(items, 0);   // chunks of each item so far, CTA by CTA
  for (unsigned c = 0; c < ctas; ++c) {
    const int count = parts(items, chunks, c, ctas);
    if (count < 1 || count > kParts) return 1;
    for (int k = count - 1; k >= 0; --k) {
      // (from the last part on: an item's end, which another CTA began, comes last)
      Run r = {};
      if (!shared_part(items, chunks, c, ctas, k, r)) return 7;
      if (r.item >= items || r.from < 0 || r.from >= r.to || r.to > (int)chunks) return 2;
      if (r.from != (int)next[r.item]) return 3;
      if (r.from > 0 && (k != count - 1 || r.to != (int)chunks)) return 4;
      if (r.to < (int)chunks && (k != 0 || c + 1 == ctas)) return 5;
      next[r.item] = (unsigned)r.to;
    }
  }
  for (unsigned n : next)
    if (n != chunks) return 6;
  return 0;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("share")
    (d / "share.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-I", wbuild.CSRC,
                    str(d / "share.cpp"), "-o", str(d / "share.so")], check=True)
    lib = ctypes.CDLL(str(d / "share.so"))
    lib.shares.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_longlong]
    return lib


def test_every_chunk_once_on_any_gpu(lib):
    seen = 0
    for sms in list(range(1, 40)) + [46, 56, 64, 78, 84, 100, 108, 114, 128, 132, 144, 148, 152, 160, 188, 192]:
        for passes in (1, 2, 3):
            for each in range(1, 22 * sms // passes + 8, 1 + sms // 40):
                if lib.shares(each * passes, passes, sms):
                    for chunks in (1, 2, 3, 8, 61):
                        assert lib.wrong(each, chunks, sms // passes) == 0, (sms, passes, each, chunks)
                        seen += 1
    assert seen > 10000


def test_runs_that_pass_the_table_are_not_shared(lib):
    """A GPU with fewer SMs than passes has no CTA for each, and one with few loses many to
    rounding: 77 items a pass on 11 SMs, 3 CTAs of 25.7 items."""
    assert not any(lib.shares(n, 3, sms) for sms in (1, 2) for n in range(3, 70, 3))
    assert max(lib.parts(77, 61, c, 3) for c in range(3)) > lib.table()
    for sms in range(3, 200):
        for passes in (1, 2, 3):
            ctas = sms // passes
            for each in range(1, 24 * ctas + 2):
                if lib.shares(each * passes, passes, sms):
                    assert max(lib.parts(each, 61, c, ctas) for c in (0, ctas // 2, ctas - 1)) <= lib.table()


def test_what_a_gb300_shares(lib):
    """152 SMs: as many items as before, and no more."""
    def rule(items, sms):
        return sms < items <= 20 * sms and -(-items // sms) * sms * 20 > items * 21
    for passes in (1, 2, 3):
        for items in range(passes, 3200, passes):
            assert bool(lib.shares(items, passes, 152)) == rule(items, 152), (passes, items)
