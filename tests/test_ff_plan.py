"""Shared memory of the small-M feed-forward kernel: the CTAs that a plan counts on an SM fit there.  The kernel's own
functions are compiled into a small host program; nothing is launched."""
import os
import shutil
import subprocess

import pytest

from tiled_dense_gemm_fp16_b200 import build

PROGRAM = """
#include <cstdio>
#include "gemm_ff_skinny.cuh"
int main() {
  using Cfg = tg::FfSkinnyCfg;
  for (int m_pad = 16; m_pad <= 256; m_pad += 16)
    for (int a_km = 0; a_km < 2; ++a_km) {
      if (a_km && m_pad % 64) continue;
      const int a = Cfg::a_bytes(m_pad, a_km), stages = Cfg::stages(m_pad, a_km);
      std::printf("%d %d %d %d %d %d\\n", m_pad, a_km, Cfg::ctas_per_sm(m_pad), stages, Cfg::W_STAGE_BYTES + a,
                  Cfg::smem_bytes(a, stages));
    }
}
"""

SM, RESERVED, CTA_MOST = 228 * 1024, 1024, 227 * 1024  # bytes of an SM, of it per resident CTA, the most a CTA may have


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    nvcc = build._nvcc()
    if not (os.path.exists(nvcc) or shutil.which(nvcc)):
        pytest.skip("no nvcc")
    where = tmp_path_factory.mktemp("plan")
    source, program = where / "plan.cu", where / "plan"
    source.write_text(PROGRAM)
    subprocess.run([nvcc, *build.ARCH, "-std=c++17", f"-I{build.CSRC}", f"-I{os.path.join(build.ROOT, 'include')}", str(source),
                    "-o", str(program)], check=True, timeout=600)
    out = subprocess.run([str(program)], check=True, capture_output=True, text=True, timeout=60).stdout
    return [tuple(int(v) for v in line.split()) for line in out.splitlines()]


def test_planned_ctas_fit(plans):
    assert len(plans) == 16 + 4
    for m_pad, a_km, per_sm, stages, stage, smem in plans:
        assert per_sm == (2 if m_pad <= 128 else 1)
        assert smem <= CTA_MOST and per_sm * (smem + RESERVED) <= SM, (m_pad, a_km, per_sm, smem)
        assert stages >= 2 and stages * stage >= m_pad * 128 * 4, (m_pad, a_km, stages)  # the partial reuses the ring


def test_rings_are_as_deep_as_fits(plans):
    for m_pad, a_km, per_sm, stages, stage, smem in plans:
        if m_pad > 32 and stages < 8:
            assert per_sm * (smem + stage + RESERVED) > SM or smem + stage > CTA_MOST, (m_pad, a_km, stages)
