"""The bench reports a kernel's measured traffic only while the kernel's sources are those that were measured."""
import os
import re

import bench
from conftest import ROOT


def test_every_header_of_the_product_kernels_counts():
    csrc = os.path.join(ROOT, "w4_dequant_gemm_amd", "csrc")
    todo, seen = [s for s in bench.KERNEL_SOURCES if s.endswith(".hip")], set()
    assert len(todo) == 4
    while todo:
        s = todo.pop()
        seen.add(s)
        with open(os.path.join(ROOT, s)) as f:
            for name in re.findall(r'^#include "([a-z_0-9]+\.hpp)"', f.read(), flags=re.M):
                rel = os.path.relpath(os.path.join(csrc, name), ROOT)
                # (launch.hpp: the host's limits of a launch, no code of a kernel)
                if rel not in seen and name != "launch.hpp":
                    todo.append(rel)
    assert seen == set(bench.KERNEL_SOURCES)
