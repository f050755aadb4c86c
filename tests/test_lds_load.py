"""The hand-written global -> LDS loads compile without a warning and leave m0,
which the compiler keeps for itself, as they found it (hipcc cross-compiles
here; no GPU needed)."""
import glob
import os
import re
import subprocess

from shared_matrix_expert_amd import build

SOURCE = """
#include "lds_load.h"
__global__ void probe(const unsigned char* p, unsigned off, unsigned dst) {
    em::lds_load16(p + 16 * threadIdx.x, dst);
    em::lds_load16(p, off * threadIdx.x, dst + 1024);
    em::lds_load4(p, off * threadIdx.x, dst + 2048);
}
"""


def test_loads_put_m0_back(tmp_path):
    src = tmp_path / "probe.hip"
    src.write_text(SOURCE)
    r = subprocess.run([build.hipcc(), *build._flags(), "-Werror=inline-asm", "-I", build.CSRC, "-S", "--cuda-device-only",
                        str(src), "-o", str(tmp_path / "probe.s")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lines = [t.strip() for t in (tmp_path / "probe.s").read_text().splitlines()]
    loads = [i for i, t in enumerate(lines) if t.startswith("global_load_lds")]
    assert len(loads) == 3
    for i in loads:
        kept = re.fullmatch(r"s_mov_b32 (s\d+), m0", lines[i - 3])
        assert kept and lines[i + 1] == f"s_mov_b32 m0, {kept.group(1)}", lines[i - 3:i + 2]


def test_no_other_asm_writes_m0():
    for path in glob.glob(os.path.join(build.CSRC, "*")):
        if os.path.basename(path) == "lds_load.h":
            continue
        text = open(path, encoding="utf-8").read()
        assert not re.search(r"s_mov_b32 m0|\"m0\"", text), path
