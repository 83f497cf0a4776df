"""The forward's two slots take turns at their exponent phases only in units
where both have the same number of them: a slot that waits for phases which the
other never has waits out its limit, in that unit and (the count is carried on)
in the ones after it.

The units are decoded on the host by the kernel's own code."""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import oracle
from flashattention_attn_fwd_gb300 import attn_fwd, sync_status, synth

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "flashattention_attn_fwd_gb300")

PROGRAM = r"""
#include <cstdio>
#include "fused_attn.cuh"

int main() {
  long apart = 0, units = 0, turns = 0;
  const int lengths[] = {1, 100, 128, 129, 300, 640, 700}, windows[] = {1, 64, 128, 129, 300}, sinks[] = {1, 4, 130, 1000};
  const int groups[] = {1, 2, 3, 5};
  for (int L : lengths) for (int w : windows) for (int sink : sinks) for (int g : groups) for (int d : {32, 64}) {
    fl::KParams p{};
    p.B = 2; p.Hkv = 2; p.Hq = 2 * g; p.group = g; p.Lq = p.Lk = L;
    p.n_qtiles = (L + 127) / 128;
    p.mask_kind = fl::MASK_WINDOW; p.window = w; p.sink = sink;
    p.slot_mode = g == 1 ? fl::SLOT_ROWS : fl::SLOT_HEADS;
    p.pairs_per_group = (g + 1) / 2;
    p.num_units = g == 1 ? p.B * p.Hq * ((p.n_qtiles + 1) / 2) : p.B * p.Hkv * p.pairs_per_group * p.n_qtiles;
    for (int u = 0; u < p.num_units; ++u) {
      const fl::SinkUnit U = fl::decode_unit<fl::KIND_ATTN, fl::SinkUnit>(p, u, true, fl::sink_skip_ok(d, d));
      const bool equal = fl::slot_len(U, 0) == fl::slot_len(U, 1);
      ++units;
      if (fl::same_tiles(U)) {
        ++turns;
        if (!equal) { std::printf("L %d window %d sink %d group %d unit %d: %d and %d tiles\n", L, w, sink, g, u,
                                  fl::slot_len(U, 0), fl::slot_len(U, 1)); return 1; }
      }
      apart += !equal && U.lo[0] == U.lo[1] && U.hi[0] == U.hi[1];  // the window's tiles alone do not tell
    }
  }
  std::printf("%ld units, %ld in turns, %ld apart\n", units, turns, apart);
  return apart > 0 && turns > 0 ? 0 : 2;
}
"""


def test_units_in_turns_have_equal_tile_counts(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src, exe = tmp_path / "turns.cu", tmp_path / "turns"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", f"-I{PKG}/csrc", f"-I{ROOT}/include",
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


@pytest.mark.gpu
@pytest.mark.parametrize("case", [(3, 1, 700, 64), (5, 1, 300, 1), (3, 3, 385, 1)], ids=str)
def test_softcap_with_sinks_and_slots_without_rows(case):
    """Odd groups and odd query tiles against the oracle.  P and the result are
    rounded to bf16, 2^-8 of at most max |v| each, and scores are off by ds = 72
    2^-22 mag + 2^-20 cap + 2^-18 with mag = sum |q k| / 8 <= 12: 2 ds < 2^-10 in the
    LSE, and 2^-7 + 2^-10 < 2^-6 of max |v| in the result."""
    Hq, Hkv, L, window = case
    q, k, v = synth.attn_inputs(40, Hq, Hkv, L, 64, seed=L)   # several units a block
    kw = dict(mask="window", window=window, sink=4, score_mod="softcap", softcap=5.0)
    out, lse = attn_fwd(*(t.to("cuda") for t in (q, k, v)), **kw)
    sync_status()
    for b in (0, 39):
        ro, rl = oracle.attention(q[b:b + 1], k[b:b + 1], v[b:b + 1], **kw)
        top = float(v[b].abs().max())
        assert np.abs(out[b:b + 1].double().cpu().numpy() - ro).max() <= 2.0 ** -6 * top
        assert np.abs(lse[b:b + 1].double().cpu().numpy() - rl).max() <= 2.0 ** -10
