"""What inline assembly leaves behind, read in the compiler's output for the sources
built here."""
import re
import subprocess

from communication_compressed_optimizer_02_amd import build

KERNEL = """
#include "layer/wide.hpp"
using namespace oba;
__global__ void k(const char* from, char* to, int32_t rows, uint32_t ld) {
  __shared__ char lds[65536];
  AheadStage<kKRow, 128, 256> s;
  s.init(threadIdx.x, 0, rows, ld);
  s.ahead(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6), from, lds);
  wait_loads();
  meet();
  to[threadIdx.x] = lds[threadIdx.x];
}
"""


def test_loads_to_lds_leave_m0_as_it_was(tmp_path):
    """m0 is reserved: the compiler knows of no clobber and may keep a value in it."""
    src, out = tmp_path / "k.hip", tmp_path / "k.s"
    src.write_text(KERNEL)
    subprocess.run([build.hipcc(), *build.HIP_FLAGS, f"-I{build.INCLUDE}", f"-I{build.CSRC}",
                    "--cuda-device-only", "-S", str(src), "-o", str(out)], check=True,
                   capture_output=True)
    blocks = [[line.strip() for line in b.splitlines() if line.strip()]
              for b in re.findall(r";;#ASMSTART\n(.*?);;#ASMEND", out.read_text(), re.S)]
    loads = [b for b in blocks if any(" lds" in line for line in b)]
    assert loads
    for b in loads:
        kept = re.fullmatch(r"s_mov_b32 (\S+), m0", b[0])
        assert kept and b[-1] == f"s_mov_b32 m0, {kept.group(1)}", b
        assert not any(re.match(rf"\S+ {kept.group(1)}\b", line) for line in b[1:]), b
    assert all("m0" not in line for b in blocks if b not in loads for line in b)
