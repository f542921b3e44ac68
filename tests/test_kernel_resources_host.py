"""What every kernel of the library takes of an SM, from ptxas's own report (nvcc
cross-compiles; no GPU needed): shared memory."""
import os
import re
import shutil
import subprocess

import pytest


def _kernel_name(mangled):
    """The kernel's own name: the last length-prefixed part of a mangled name."""
    at = mangled.index("_ZN") + 3 if "_ZN" in mangled else 2
    name = None
    while at < len(mangled) and mangled[at].isdigit():
        digits = re.match(r"\d+", mangled[at:]).group(0)
        at += len(digits)
        name, at = mangled[at:at + int(digits)], at + int(digits)
    return name


def _template_arguments(mangled):
    return tuple(int(x) for x in re.findall(r"L[ib](\d+)E", mangled))


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """[(name, template arguments, registers, static shared memory)] of both units."""
    from spacetime_attention_vdit_b200 import build
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    folder = tmp_path_factory.mktemp("resources")
    objects = [str(folder / (os.path.basename(src) + ".o")) for src in build.OBJECT_SOURCES]
    commands = [build.object_command(src, obj, ptxas_verbose=True) for src, obj in zip(build.OBJECT_SOURCES, objects)]
    commands.append(build.command(ptxas_verbose=True, out=str(folder / "lib.so"), objects=objects))
    out, mangled = [], None
    for cmd in commands:
        res = subprocess.run(cmd, capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-2000:]
        for line in res.stderr.splitlines():
            m = re.search(r"Compiling entry function '(\w+)'", line)
            if m:
                mangled = m.group(1)
            m = re.search(r"Used (\d+) registers", line)
            if m and mangled:
                smem = re.search(r"(\d+) bytes smem", line)
                out.append((_kernel_name(mangled), _template_arguments(mangled), int(m.group(1)),
                            int(smem.group(1)) if smem else 0))
                mangled = None
    assert len(out) > 40
    return out


def test_names_are_read_whole():
    assert _kernel_name("_ZN4vdit25bwd_qk_norm_rope3d_kernelILb0ELi4EEEvNS_13NormBwdParamsE") == "bwd_qk_norm_rope3d_kernel"
    assert _template_arguments("_ZN4vdit25bwd_qk_norm_rope3d_kernelILb0ELi4EEEvNS_13NormBwdParamsE") == (0, 4)
    assert _kernel_name("_ZN4vdit48_GLOBAL__N__7d585335_15_block_select_cu_13bcb03b17block_pick_kernelILi4EEEvPKj") == "block_pick_kernel"


def test_two_norm_rope_ctas_fit_an_sm(kernels):
    """Dynamic shared memory starts behind a kernel's static variables, at its own
    alignment.  The norm + rotation pass runs two CTAs per SM at width 5,120 (a ring of
    81,920 bytes, its small variables, 8 bytes per table entry) with up to 3,952
    entries; padding would take the second one from 3,841 on."""
    from spacetime_attention_vdit_b200 import build
    source = open(os.path.join(build.CSRC, "patchify_rope.cuh")).read()
    stages, pairs = (int(re.search(rf"constexpr int {name} = (\d+)", source).group(1))
                     for name in ("kNormStages", "kRopeMaxPairs"))
    held = -(-(2 * 4 * 4 + 2 * pairs * 8 + stages * 8) // 128) * 128 if "kNormHeadBytes" in source else 0
    found = [smem for name, _, _, smem in kernels if name == "qk_norm_rope3d_kernel"]
    assert len(found) == 2
    for static in found:
        cta = 1024 + static + held + stages * 2 * 5120 * 2 + 3952 * 8    # the system keeps 1 KB of each CTA
        assert 2 * cta <= 228 * 1024, (static, held)
