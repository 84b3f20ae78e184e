"""The compiled 256 x 256 product kernels: no inline-asm MFMA result is read before its latency has passed, and no
accumulator or fragment is written by a vector instruction right before an inline-asm MFMA that reads it; the main
loops neither spill nor wait for every load under way."""

from __future__ import annotations

import importlib.util
import os
import re
import shutil
import subprocess

import pytest

from test_isa_mfma_latency import CSRC, ROOT, early_reads


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    hipcc = shutil.which("hipcc") or ("/opt/rocm/bin/hipcc" if os.path.exists("/opt/rocm/bin/hipcc") else None)
    if hipcc is None:
        pytest.skip("hipcc is not available")
    spec = importlib.util.spec_from_file_location("_muon_build", os.path.join(ROOT, "muon_newton_schulz_step_amd", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    out = str(tmp_path_factory.mktemp("isa") / "k_linear256.s")
    cmd = [hipcc, *build.COMMON, "--cuda-device-only", "-S", os.path.join(CSRC, "k_linear256.hip"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    return open(out).read()


def test_no_asm_mfma_result_is_read_early(listing):
    assert len(re.findall(r";;#ASMSTART\s*\n\s*v_mfma", listing)) > 0
    bad = early_reads(listing)
    assert bad == [], f"{len(bad)} early reads, e.g. {bad[:5]}"


def main_loops(listing):
    """The innermost loops with 128 MFMAs, one a kernel."""
    for m in re.finditer(r"^(_ZN\S*kl_linear256\S*):(.*?)^\.Lfunc_end", listing, re.S | re.M):
        lines = m.group(2).split("\n")
        labels = {x.group(1): i for i, line in enumerate(lines) if (x := re.match(r"(\.LBB\S+):", line))}
        for i, line in enumerate(lines):
            b = re.match(r"\s+s_c?branch\S*\s+(\.LBB\S+)", line)
            if b and labels.get(b.group(1), i) < i:
                body = lines[labels[b.group(1)]:i]
                if sum("v_mfma" in x for x in body) == 128:
                    yield m.group(1), body
                    break


def test_main_loops_keep_loads_under_way(listing):
    loops = list(main_loops(listing))
    assert len(loops) == 6
    for name, body in loops:
        waits = [x.strip() for x in body if "vmcnt" in x]
        assert waits == ["s_waitcnt vmcnt(6)"], (name, waits)
        assert not any("scratch_" in x or "v_accvgpr" in x for x in body), name
        assert sum("buffer_load_dwordx4" in x and "lds" in x for x in body) == 16, name
