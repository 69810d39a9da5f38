"""Refusals of the serving entry points that need no GPU, and the turns-per-position of the rotation."""
import math
import subprocess
from pathlib import Path

import decode_attention_host_b200 as dkv

ROOT = Path(__file__).resolve().parent.parent


def test_null_handles_are_rejected():
    lib, none = dkv.lib, None
    assert lib.dkv_extend_tables(none, none, none, 1, none, 1, none, 0, none, none, none, none, 0, none) \
        == dkv.DKV_ERR_INVALID_ARG
    assert lib.dkv_store_kv(none, none, none, 0, none, 1, 0, none, none, none, none, none, 0) \
        == dkv.DKV_ERR_INVALID_ARG
    assert lib.dkv_attn_chunk(none, none, 0, none, 1, none, none, none, none, none, none, 0, none, 0, 0, 1, none, 1, 1,
                              0, none, none) == dkv.DKV_ERR_INVALID_ARG
    assert lib.dkv_attn_decode_window(none, 1, 0, 0, none, none, none, none, none, none, none, 0, none, none, 1, 1, 0) \
        == dkv.DKV_ERR_INVALID_ARG
    assert "null handle" in dkv.dkv_last_error_string()


def test_turns_per_position_match_the_angles(tmp_path):
    """p * turns mod 2^64 is the angle of position p as a fraction of a turn: against exact rational arithmetic
    on the same double frequency, within (p + 1) * 2^-64 turns and the rounding of the division by 2 pi."""
    src = tmp_path / "turns.cpp"
    src.write_text("""
#include <cstdio>
#include <initializer_list>
#include "dkv_plan.h"
int main() {
  for (double base : {1e4, 5e5, 0.0})
    for (int D : {64, 128}) {
      double f[64]; uint64_t t[64];
      dkv::rope_frequencies(base, D, f);
      dkv::rope_turns(f, D, t);
      for (int i = 0; i < D / 2; ++i) printf("%a %llu\\n", f[i], (unsigned long long)t[i]);
    }
}
""")
    exe = tmp_path / "turns"
    subprocess.run(["g++", "-std=c++17", f"-I{ROOT}/decode_attention_host_b200/csrc", "-o", str(exe), str(src)],
                   check=True)
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
    from fractions import Fraction
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    seen = 0
    for line in filter(None, lines):
        f, t = line.split()
        freq, turns = Fraction(float.fromhex(f)), int(t)
        for pos in (0, 1, 127, 4096, 2 ** 20 + 3, 2 ** 30 - 1):
            exact = freq * pos / two_pi
            got = Fraction(pos * turns % 2 ** 64, 2 ** 64)
            diff = abs((got - exact + Fraction(1, 2)) % 1 - Fraction(1, 2))
            # one step of the stored fraction and the long double quotient (2^-63 relative) a position
            assert diff <= Fraction(pos + 1, 2 ** 62), (f, pos)
            seen += 1
    assert seen == 6 * (32 + 64) * 3 and math.isclose(float(two_pi), 2 * math.pi)


def test_even_split_plan_covers_every_block_and_stays_in_the_workspace(tmp_path):
    """plan_split_even on a grid of sizes: every block in some split, no split empty, never fewer splits than the
    plain plan and never more than 16 beyond it or max_nsplit, and no costlier plan than the plain one."""
    src = tmp_path / "plan.cpp"
    src.write_text(r"""
#include <cstdio>
#include <initializer_list>
#include "dkv_plan.h"
int main() {
  long n = 0;
  for (int bs : {16, 48, 256, 1024})
    for (int nblk : {1, 2, 3, 17, 66, 259, 2048, 65536})
      for (long per : {1L, 3L, 8L, 512L, 2048L, 100000L})
        for (long warps : {1184L, 1776L, 4736L})
          for (long cap : {1L, 7L, 40L, 100000L}) {
            const dkv::SplitPlan a = dkv::plan_split(nblk, per, bs, warps, 0);
            const dkv::SplitPlan b = dkv::plan_split_even(nblk, per, bs, warps, cap);
            auto cost = [&](const dkv::SplitPlan& s) {
              return static_cast<double>((per * s.nsplit + warps - 1) / warps) * (static_cast<double>(s.bps) * bs + 48);
            };
            if (static_cast<long>(b.nsplit) * b.bps < nblk || static_cast<long>(b.nsplit - 1) * b.bps >= nblk) return 1;
            if (b.nsplit < a.nsplit || b.nsplit > a.nsplit + 16) return 2;
            if (b.nsplit > a.nsplit && b.nsplit > cap) return 3;
            if (cost(b) > cost(a)) return 4;
            ++n;
          }
  printf("%ld\n", n);
  // 64 sequences of 8 kv heads, 259 visible blocks of 16: four nearly full rounds of 9 splits
  return dkv::plan_split_even(259, 512, 16, 1184, 1 << 20).nsplit == 9 ? 0 : 5;
}
""")
    exe = tmp_path / "plan"
    subprocess.run(["g++", "-std=c++17", f"-I{ROOT}/decode_attention_host_b200/csrc", "-o", str(exe), str(src)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.returncode
