"""What the compiler gives the kernels whose launches count on it (registers, spills), from its own
report; no GPU."""
import os
import re
import shutil
import subprocess

import pytest

from orthogonal_reparameterized_cnp_b200 import build


def _report(source, kernel):
    """(template arguments, registers, spilled bytes) of every instance of `kernel` in `source`."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    r = subprocess.run([nvcc, *build.NVCC_FLAGS, "-Xptxas", "-v", "-c",
                        os.path.join(build.CSRC, source), "-o", os.devnull],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    got = []
    for part in r.stderr.split("Compiling entry function '")[1:]:
        name = re.match(rf"\w*?\d{kernel}I(\w*?)EEv", part)
        if name:
            args = re.findall(r"L\w(\d+)E|([a-z])", name.group(1) + "E")
            got.append((tuple(int(n) if n else t for n, t in args),
                        int(re.search(r"Used (\d+) registers", part).group(1)),
                        int(re.search(r"(\d+) bytes spill stores", part).group(1))))
    return got


def test_wide_merge_runs_two_blocks_on_a_multiprocessor():
    """Rows of more than 8192 columns (four code words a thread): blocks of up to 512 threads of
    which two run at once, in 65536 registers, spilling 32 words at most."""
    got = _report("kernels_q4.cu", "k_merge_q4_pairs")
    wide = [g for g in got if g[0][2] == 4]
    assert len(got) == 18 and len(wide) == 6  # (types x groups x words a thread)
    for args, registers, spilled in wide:
        assert 2 * 512 * registers <= 65536 and spilled <= 4 * 32, (args, registers, spilled)


def test_products_of_tens_of_tokens_keep_their_values_in_registers():
    """No spills in any token tile, in either direction."""
    got = _report("kernels_umma_q4.cu", "k_umma_q4")
    assert len(got) == 9  # (tiles of 32 .. 256 tokens, of 16 transposed only)
    assert [g for g in got if g[2]] == []
