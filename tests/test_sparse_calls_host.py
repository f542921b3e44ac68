"""Host-side checks of how the sparse-attention and gradient calls reach the
device (no GPU needed): the stream they launch on, what they refuse, and what
their kernels may not do."""
import contextlib
import os
import re

import pytest
import torch

from tests.test_abi_host import ALIGN, FAKE, L, SHAPE  # noqa: F401  (L: fixture)
from tests.test_sparse_host import _Pretend, norm_bwd, select


@pytest.mark.parametrize("handle,want", [(0, 0), (1, 1), (0x7f00, 0x7f00)])
def test_a_stream_handle_launches_on_that_stream(monkeypatch, handle, want):
    """Handle 0 is the default stream.  torch takes an ExternalStream of 0 for one
    without a handle and makes a stream of its own, on which the kernels would run
    beside the work that produces their inputs."""
    import spacetime_attention_vdit_b200 as vd

    class Stream:
        def __init__(self, cuda_stream):
            self.cuda_stream = cuda_stream

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h: Stream(h if h else 0xbad))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "stream", contextlib.nullcontext)
    context, got = vd._launch_stream(_Pretend(1, 200, 2, 32), "q", handle)
    assert got == want
    with context as st:
        assert st.cuda_stream == want            # what the call allocates belongs to the same stream


def _sources():
    from spacetime_attention_vdit_b200 import build
    return {name: re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, name)).read())
            for name in sorted(os.listdir(build.CSRC)) if name.endswith((".cu", ".cuh", ".h"))}


def _kernels():
    """{name: (parameter list, body)} of every kernel in the sources, comments gone."""
    out = {}
    for text in _sources().values():
        for m in re.finditer(r"__global__ void\s+(?:__launch_bounds__\([^{;]*?\)\s+)?(\w+)\s*\(", text):
            at, depth = m.end(), 1
            while depth:
                depth += {"(": 1, ")": -1}.get(text[at], 0)
                at += 1
            params, begin = text[m.end():at - 1], text.index("{", at)
            end, depth = begin + 1, 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            out[m.group(1)] = (params, text[begin + 1:end - 1])
    return out


def _launched_early():
    """Names of the kernels that launch_early() starts, through a variable too."""
    names, kernels = set(), _kernels()
    for text in _sources().values():
        for m in re.finditer(r"launch_early\((\w+),", text):
            name = m.group(1)
            if name in kernels:
                names.add(name)
                continue
            held = re.search(rf"auto {name} =([^;]*);", text)
            assert held, name
            picked = set(re.findall(r"\b(\w+_kernel)\b", held.group(1)))
            assert picked and picked <= set(kernels)
            names |= picked
    return names


def test_kernels_launched_early_wait_before_they_read_or_leave():
    """A kernel that may start before its predecessor has finished waits for it
    first: before any return (the next kernel of the stream waits for this one
    alone) and before it reads the watchdog's flag or memory."""
    kernels, early = _kernels(), _launched_early()
    assert {"block_scores_kernel", "block_pick_kernel", "bwd_weights_qk_norm_rope3d_kernel"} <= early
    for name in early:
        before, found, _ = kernels[name][1].partition("wait_for_previous();")
        assert found, name
        for statement in before.split(";"):
            words = statement.split()
            assert not words or words[0] in ("__shared__", "let_next_start()"), (name, statement)


def test_kernels_launched_early_read_coherently():
    """Memory that the previous kernel may still be writing when this one starts is
    not read-only for its lifetime: no non-coherent loads, and no __restrict__ that
    would let the compiler use them."""
    kernels = _kernels()
    for name in _launched_early():
        params, body = kernels[name]
        assert "__restrict__" not in params, name
        assert "__ldg" not in body and "ld.global.nc" not in body and "__restrict__" not in body, name


def test_weight_gradients_are_checked_for_alignment(L):  # noqa: F811
    """dwq and dwk are written as float32: an address between two of them is refused."""
    for name in ("dwq", "dwk"):
        assert norm_bwd(L, **{name: FAKE + 2}) == ALIGN
        assert norm_bwd(L, **{name: FAKE + 1}) == ALIGN


def test_watchdog_sites_are_told_apart():
    """A timeout reports the number of its wait alone: no two waits of different
    kernels may have one number, and it has to fit its 8 bits."""
    sites, literal = {}, set()
    for name, text in _sources().items():
        for body in re.findall(r"enum : int \{([^}]*)\}", text) + re.findall(r"constexpr int (kSite[^;]*);", text):
            if "kSite" not in body:
                continue
            value = -1
            for item in body.split(","):
                key, _, given = (x.strip() for x in item.partition("="))
                value = int(given) if given else value + 1
                assert key not in sites, key
                sites[key] = value
        literal |= {int(x) for x in re.findall(r"(?:mbar_wait|warp_wait|mbar_drain_site)\([^;]*?, (\d+)\)\)", text)}
        literal |= {int(x) for x in re.findall(r"watchdog_trip\((\d+)\)", text)}
    assert len(sites) > 20 and literal
    values = list(sites.values()) + sorted(literal)
    assert len(set(values)) == len(values), sorted((v, k) for k, v in sites.items() if values.count(v) > 1)
    assert all(0 < v < 256 for v in values)


def test_the_selections_limits_are_the_headers(L):  # noqa: F811
    """Sizes past the launch grid are refused as the header says, before any launch."""
    from tests.conftest import ROOT
    assert select(L, B=1, heads=65536, Lq=1, Lk=1, D=32, top_k=1) == SHAPE
    assert select(L, B=65536, heads=1, Lq=1, Lk=1, D=32, top_k=1) == SHAPE
    assert select(L, B=256, heads=256, Lq=1, Lk=1, D=32, top_k=1) == SHAPE
    assert select(L, heads=1, Lq=536_862_721, D=32) == SHAPE
    header = re.sub(r"\s*\n \* ?", " ", open(os.path.join(ROOT, "include", "vdit.h")).read())
    text = header[header.index("vdit_attn_select_blocks - "):header.index("int vdit_attn_select_blocks(")]
    assert "B * heads above 65,535" in text and "Lq above 536,862,720" in text
