"""The device code of the products' hand-placed DMA under the library's own
build flags."""

import os
import re
import shutil
import subprocess

import pytest

from bit_quantized_moe_token_amd import build

PROGRAM = """
#include "gemm.hpp"
using namespace moeq;
__global__ void transfers(i32x4 rs, uint32_t voff, uint32_t soff) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  lds_dma_raw<16>(rs, voff * threadIdx.x, soff, lds);
  lds_dma_raw<4>(rs, voff * threadIdx.x, soff, lds + 1024);
  vm_wait<0>();
}
"""


@pytest.mark.skipif(not os.path.exists(build.HIPCC) and not shutil.which(build.HIPCC), reason="no compiler")
def test_reserved_registers_keep_their_value(tmp_path):
    """m0, which holds a transfer's LDS address, is written by the compiler
    alone: no asm writes it or lists it as clobbered (of which the compiler
    warns; the build silences nothing)."""
    src, out = tmp_path / "transfers.hip", tmp_path / "transfers.s"
    src.write_text(PROGRAM)
    flags = build.CFLAGS + build.FILE_FLAGS["gemm_f16.hip"]
    assert not [f for flags_of in build.FILE_FLAGS.values() for f in flags_of if f.startswith("-Wno-")]
    r = subprocess.run([build.HIPCC, *flags, "-S", "--cuda-device-only", "-I", build.CSRC, str(src), "-o", str(out)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "reserved register" not in r.stderr
    blocks = re.findall(r"#ASMSTART(.*?)#ASMEND", out.read_text(), re.S)
    blocks = [[l.strip() for l in b.splitlines() if l.strip() and l.strip()[0] not in ";#"] for b in blocks
              if "lds" in b]
    assert len(blocks) == 2
    for b in blocks:
        assert not any(re.match(r"\S+ m0\b", l) for l in b)
    assert len(re.findall(r"^\s*s_\w+ m0,", out.read_text(), re.M)) >= 2


@pytest.mark.skipif(not os.path.exists(build.HIPCC) and not shutil.which(build.HIPCC), reason="no compiler")
def test_norms_use_no_scratch():
    """The norms' kernels hold their rows and sums in registers: the compiler
    reports no scratch for any of them."""
    src = os.path.join(build.CSRC, "norm.hip")
    r = subprocess.run([build.HIPCC, *build.CFLAGS, "-Rpass-analysis=kernel-resource-usage", "-S", "--cuda-device-only", src,
                        "-o", os.devnull], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    found = re.findall(r"Function Name: (\S+).*?ScratchSize \[bytes/lane\]: (\d+)", r.stderr, re.S)
    assert len(found) > 60
    assert not [name for name, size in found if int(size)]
