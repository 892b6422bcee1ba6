"""The listing of the built library: waits that no result shows reliably."""
import os
import re
import shutil
import subprocess

import pytest

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


@pytest.fixture(scope="module")
def functions(tmp_path_factory):
    """Kernels of libw4.so by name, as lists of instructions."""
    import w4_dequant_gemm_amd as w4
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    if not os.path.exists(w4.library_path):
        from w4_dequant_gemm_amd import build
        build.build()
    folder = tmp_path_factory.mktemp("listing")
    shutil.copy(w4.library_path, folder / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=folder, check=True, capture_output=True)
    found = {}
    for name in sorted(os.listdir(folder)):
        if not name.endswith("gfx950"):
            continue
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", name], cwd=folder, check=True,
                              capture_output=True, text=True).stdout
        for line in text.splitlines():
            head = re.match(r"(?:[0-9a-f]+ )?<(.+)>:$", line)
            if head:
                body = found.setdefault((name, head.group(1)), [])
            elif line.startswith("\t"):
                body.append(line.split("//")[0].strip())
    return found


def test_loads_to_shared_memory_wait_for_m0(functions):
    """A load to shared memory takes its place from M0, and needs a wait state behind the scalar instruction that
    writes M0.  The compiler keeps that where it places both; inside an asm statement it does not look."""
    loads = 0
    for (_, name), body in functions.items():
        for before, now in zip(body, body[1:]):
            if re.match(r"(global|scratch)_load_lds_|buffer_load_.*\blds\b", now):
                loads += 1
                assert not re.match(r"s_\w+ m0,", before), (name, before, now)
    assert loads > 100                       # the tiled products and attention
