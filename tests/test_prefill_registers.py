"""The dense prefill kernel of 128 channels in bf16 has two thread blocks of 224 threads an SM, 128 registers a
thread, all of which it uses: a spill costs it 2.6 %.  What the compiler says of it (no GPU needed)."""

import os
import re
import subprocess

from paged_kv_cache_317_gb300 import _build


def test_the_dense_prefill_kernel_does_not_spill(tmp_path):
    said = subprocess.run([_build.nvcc_path(), *_build.ARCH, *_build.FLAGS, "-Xptxas", "-v", "-c",
                           os.path.join(_build.CSRC, "paged_prefill.cu"), "-o", str(tmp_path / "prefill.o")],
                          capture_output=True, text=True, check=True).stderr
    # the instance of <bf16, 128 channels, dense, two numbers a probability>
    entry = re.search(r"paged_prefill_kernelILb1ELi128ELb0ELb0E.*?(\d+) bytes spill stores, (\d+) bytes spill loads"
                      r".*?Used (\d+) registers", said, re.S)
    assert entry and [int(n) for n in entry.groups()] == [0, 0, 128]
