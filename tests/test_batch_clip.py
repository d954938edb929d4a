"""The cut of a batch's lengths (csrc/batch_clip.h, what the kernels of the cache
compute addresses from) over the corners of its arguments, on the host."""
import os
import subprocess

import pytest

from helpers import ROOT

PROGRAM = r"""
#include <climits>
#include <cstdint>
#include <cstdio>
#include "batch_clip.h"

int main() {
  const int some[] = {INT_MIN, INT_MIN + 1, INT_MIN + 5, INT_MIN / 2, -100, -5, -1, 0, 1, 2, 5, 7, 99, 100, 101,
                      (1 << 24) - 1, 1 << 24, (1 << 24) + 1, 1 << 30, (1 << 30) + 1, INT_MAX - 5, INT_MAX - 1, INT_MAX};
  const int tokens[] = {1, 7, 100, 1 << 24}, mosts[] = {8, 100, 1 << 30};
  int wrong = 0;
  for (int lo : some) for (int hi : some) for (int ctx : some) for (int T : tokens) for (int most : mosts) {
    const moex::SeqView s = moex::clip_seq(lo, hi, ctx, T, most);
    const int64_t end = static_cast<int64_t>(s.first) + s.n;
    const bool fine = lo >= 0 && lo <= hi && hi <= T && ctx >= 0 && ctx <= most;
    bool ok = s.first >= 0 && s.n >= 0 && end <= T && s.ctx >= 0 && s.ctx <= most && s.bad == !fine;
    if (fine) ok = ok && s.first == lo && s.n == hi - lo && s.ctx == ctx;
    if (!ok && ++wrong <= 5) std::printf("%d %d %d of %d, %d: %d + %d, %d, bad %d\n", lo, hi, ctx, T, most, s.first, s.n, s.ctx, s.bad);
  }
  std::printf("%d wrong\n", wrong);
  return wrong != 0;
}
"""


def test_lengths_are_cut_to_the_batch(tmp_path):
    src, exe = tmp_path / "clip.cpp", tmp_path / "clip"
    src.write_text(PROGRAM)
    # -fwrapv: where 32 bits are left, what the GPU would compute
    cmd = [os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-fwrapv", "-I" + os.path.join(ROOT, "moe_expert_gb300", "csrc"),
           str(src), "-o", str(exe)]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


@pytest.mark.gpu
@pytest.mark.parametrize("n", [[3, 4, 2], [60, 50, 40]])
@pytest.mark.parametrize("corrupt", [(1, -(1 << 31) + 5), (2, -(1 << 31)), (1, (1 << 31) - 1), (0, -(1 << 31)), (3, -1)])
def test_corrupt_offsets_touch_nothing_outside(n, corrupt):
    import torch
    from layer_cases import Paged, mx, status
    from test_gpu_paged_attention import _q
    m = mx()
    p = Paged(71, n, [x + 90 for x in n], 2, 64, 16)
    q = _q(p, 4)
    good = m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q)
    cu = p.cu.clone()
    cu[corrupt[0]] = corrupt[1]
    around = torch.full((p.T + 200, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.T + 200, 4), 5.0, device="cuda")
    mine = slice(100, 100 + p.T)
    m.paged_attention(q, p.k, p.v, cu, p.ctx, p.table, max_q=p.max_q, out=around[mine], lse=lse[mine])
    assert status() == 16
    for t in (around, lse):
        assert (t[:100] == 5).all() and (t[100 + p.T:] == 5).all()
    k, v = p.k.clone(), p.v.clone()
    m.rope_kv_write(torch.zeros(p.T, 8 * 64, device="cuda"), k, v, cu, p.ctx, p.table, n_heads=4)
    assert status() == 16
    assert torch.equal(m.paged_attention(q, p.k, p.v, *p.batch(), max_q=p.max_q), good) and status() == 0
