"""Register budgets of the bounded cache's kernels, checked at compile time
(see test_build_host.py): spills, and the residency each launch counts on. Two
kernels at a register ceiling that their residency sets spill a few values
(k_prefill_stream: ten warps, three of them on one of the SM's four parts;
k_rope_axes<8>: three CTAs); both measured faster than with fewer threads."""
import concurrent.futures as cf
import os
import re

import pytest

from hybrid_local_global_b200 import build

from test_build_host import _ptxas_report

# (pattern in the mangled name, instances, most registers a thread, most spilled bytes stored or loaded)
BUDGETS = [
    (r"k_prefill_streamE", 1, 168, 32),
    (r"k_decode_sinksILi\d+ELi1E", 2, 255, 0),
    (r"k_decode_sinksILi\d+ELi2E", 2, 144, 0),  # two CTAs of 224 threads per SM
    (r"k_rope_axesILi\d+E", 2, 80, 48),          # three CTAs of 256
    (r"k_pages_copyILi\d+E", 2, 64, 0),
    (r"k_pages_(fork|trim)E", 2, 64, 0),
    (r"k_pages_(reserve|compact)E", 2, 64, 0),  # 1024 threads
    (r"k_pages_reserve_smallILi\d+E", 1, 64, 0),
]


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not os.path.exists(build.NVCC):
        pytest.skip("nvcc not found")
    names = ("prefill_stream.cu", "decode_sinks.cu", "pages.cu", "rope_axes.cu")
    files = [s for s in build.sources() if os.path.basename(s) in names]
    assert len(files) == len(names)
    out = str(tmp_path_factory.mktemp("ptxas"))
    merged = {}
    with cf.ThreadPoolExecutor(max_workers=4) as ex:
        for part in ex.map(lambda s: _ptxas_report(s, out), files):
            merged.update(part)
    return merged


@pytest.mark.parametrize("pattern,instances,regs,spill", BUDGETS)
def test_registers_and_spills(kernels, pattern, instances, regs, spill):
    found = {k: v for k, v in kernels.items() if re.search(pattern, k)}
    assert len(found) == instances, sorted(found)
    for name, v in found.items():
        assert max(v["st"], v["ld"]) <= spill and v["regs"] <= regs, (name, v)
