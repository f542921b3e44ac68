"""What every kernel of the library takes of an SM, from ptxas's own report (nvcc
cross-compiles; no GPU needed): registers and shared memory."""
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


def _source(name):
    from spacetime_attention_vdit_b200 import build
    return open(os.path.join(build.CSRC, name)).read()


def _norm_bwd_threads(v):
    three, two, one = (int(x) for x in re.search(
        r"norm_bwd_threads\(int V\) \{ return V >= 3 \? (\d+) : \(V == 2 \? (\d+) : (\d+)\); \}",
        _source("norm_rope_bwd.cuh")).groups())
    return three if v >= 3 else two if v == 2 else one


def _time_threads(d, rows):
    """The short time pass's own sum: a producer warp, and one or two warps per stage."""
    warps = 2 if (rows + 15) // 16 * 16 >= 32 else 1
    stage = 3 * rows * d * 2
    stages = min((231424 // (stage + 16)) & ~1, 16, 2 * ((10 if d >= 128 else 16) // warps))
    return 32 * (1 + stages // 2 * warps)


SPLIT = {"attn_fwd_tcgen05_kernel": ("attn_tcgen05.cuh", r"REGS_SOFTMAX = (\d+), REGS_CONTROL = (\d+)"),
         "attn_fwd_tcgen05_rope_q_kernel": ("attn_tcgen05.cuh", r"REGS_SOFTMAX = (\d+), REGS_CONTROL = (\d+)"),
         "attn_fwd_tcgen05_sparse_kernel": ("attn_block_sparse.cuh", r"REGS_SOFT = (\d+), REGS_CTRL = (\d+)"),
         "grad_attn_fwd_tcgen05_sparse_dq_kernel": ("attn_block_sparse_bwd.cuh",
                                                    r"REGS_ELEMENT = (\d+), REGS_CTRL = (\d+)"),
         "grad_attn_fwd_tcgen05_sparse_dkv_kernel": ("attn_block_sparse_bwd.cuh",
                                                     r"REGS_ELEMENT = (\d+), REGS_CTRL = (\d+)")}
# threads of each kernel's largest CTA, by exact name
THREADS = {**{name: lambda *_: 384 for name in SPLIT}, "attn_time_short_kernel": _time_threads,
           "rope3d_kernel": lambda *_: 256, "rope3d_table_kernel": lambda *_: 256, "qk_norm_rope3d_kernel": lambda *_: 256,
           "patchify3d_kernel": lambda *_: 256, "patchify122_f32_kernel": lambda *_: 128,
           "unpatchify3d_kernel": lambda *_: 256, "patch_embed_kernel": lambda *_: 320,
           "watchdog_selftest_kernel": lambda *_: 32,
           "bwd_qk_norm_rope3d_kernel": lambda wide, v: _norm_bwd_threads(v),
           "bwd_weights_qk_norm_rope3d_kernel": lambda *_: 1024, "block_means_kernel": lambda *_: 256,
           "block_scores_kernel": lambda *_: 128, "block_pick_kernel": lambda *_: 256}


def test_every_kernel_has_the_registers_for_its_largest_cta(kernels):
    """Registers of a CTA's warps fit the 16,384 of each of the SM's four
    sub-partitions (warps are spread round-robin, registers granted in multiples of
    8), so that no launch can fail for lack of them.  A kernel that is not listed
    fails, and so does a list entry that no kernel answers to."""
    assert {name for name, *_ in kernels} == set(THREADS)
    for name, arguments, registers, _ in kernels:
        threads = THREADS[name](*arguments)
        warps = -(-threads // 32)
        assert -(-warps // 4) * 32 * (-(-registers // 8) * 8) <= 16384, (name, arguments, registers, threads)


def test_launch_bounds_are_the_listed_threads():
    """The listed thread counts against the sources' launch bounds."""
    from spacetime_attention_vdit_b200 import build
    text = "\n".join(re.sub(r"//[^\n]*", "", _source(f)) for f in sorted(os.listdir(build.CSRC)))
    found = {name: bound.split(",")[0].strip() for bound, name in
             re.findall(r"__launch_bounds__\(((?:[^()]|\([^()]*\))*)\)\s+(\w+)\s*\(", text)}
    assert set(SPLIT) <= set(found) and {"block_scores_kernel", "bwd_weights_qk_norm_rope3d_kernel"} <= set(found)
    for name, bound in found.items():
        if name == "bwd_qk_norm_rope3d_kernel":
            assert bound == "norm_bwd_threads(V)"
        elif name != "attn_time_short_kernel":
            value = int(bound) if bound.isdigit() else int(re.search(rf"constexpr int {bound} = (\d+)", text).group(1))
            assert THREADS[name](0, 0) == value, (name, bound)


def test_register_splits_fit_what_the_launch_has(kernels):
    """Two warpgroups that raise their share and one that lowers its own (setmaxnreg):
    the sum is within the CTA's registers at launch, and one warp of each within a
    sub-partition's."""
    launch = int(re.search(r"REGS_LAUNCH = (\d+)", _source("attn_tcgen05.cuh")).group(1))
    for name, (source, pattern) in SPLIT.items():
        more, less = (int(x) for x in re.search(pattern, _source(source)).groups())
        assert more % 8 == 0 and less % 8 == 0
        assert 2 * 128 * more + 128 * less <= 384 * launch
        assert 32 * (2 * more + less) <= 16384
        used = {registers for n, _, registers, _ in kernels if n == name}
        assert used == {launch}, (name, used)
