"""Kernels that are set up while the one before them runs: each waits for it before it touches global memory, and
lets the next one begin only then."""
import os
import re

import pytest

from transformer_layer_decode_gb300 import build as tld_build

FILES = ["kv_rows.cu", "kv_write8.cu", "kv_attention.cu", "kv_pages.cu", "rope.cu"]


def kernels(text):
    """{name: body} of the kernels of a source file."""
    out = {}
    for m in re.finditer(r"__global__ void[^;{]*?(\w+)\((?:[^(){}]|\([^()]*\))*\)\s*\{", text):
        name = re.findall(r"(\w+)\((?:const __grid_constant__|const int32_t|int32_t|KvView|const T|T\*)", m.group(0))[-1]
        out[name] = text[m.end():text.index("\n}\n", m.end())]
    return out


def launched_behind(text):
    """Kernels launched with a configuration that lets them begin early."""
    names = set(re.findall(r"launch_after\((\w+)", text))
    for m in re.finditer(r"const BehindLast behind\(&cfg\);(.*?)\n}\n", text, re.S):
        names |= set(re.findall(r"\b(\w+)\b", m.group(1)))
    return names & set(kernels(text))


@pytest.mark.parametrize("name", FILES)
def test_every_kernel_waits_first(name):
    with open(os.path.join(tld_build.CSRC, name)) as f:
        text = f.read()
    bodies = kernels(text)
    behind = launched_behind(text)
    assert behind, "no kernel found"
    for k in sorted(behind):
        lines = [re.sub(r"//.*", "", x).rstrip() for x in bodies[k].split("\n")]
        at = [i for i, x in enumerate(lines) if "pdl_wait()" in x]
        assert len(at) == 1 and lines[at[0]] == "  pdl_wait();", (k, "one wait, of every thread")
        for x in lines[:at[0]]:  # declarations, and numbers made of the arguments
            assert re.match(r"\s*(extern )?__shared__|\s*(using|constexpr|static_assert)\b|\s*const (int|int64_t|bool) |"
                            r"\s*const KvView& c = p\.c;|\s*std::conditional_t<.*> c = view;|\s*$", x), (k, x)
            assert "[" not in re.sub(r".*__shared__.*", "", x), (k, x)
        trigger = [i for i, x in enumerate(lines) if "pdl_trigger()" in x]
        assert all(i > at[0] for i in trigger), (k, "the next kernel may begin before this one has waited")


def test_the_kernels_are_found():
    """(the sources are read as text: a kernel that the patterns above miss would go unlooked at)"""
    found = {}
    for name in FILES:
        with open(os.path.join(tld_build.CSRC, name)) as f:
            text = f.read()
        assert len(kernels(text)) == text.count("__global__ void"), (name, sorted(kernels(text)))
        found[name] = launched_behind(text)
    assert found["kv_rows.cu"] >= {"kv_rows", "kv_rows_rotated"}
    assert found["kv_write8.cu"] == {"kv_owners", "write_rows", "write_blocks"}
    assert found["kv_attention.cu"] == {"kv_attn", "kv_attn_whole", "kv_attn_join"}
    assert found["kv_pages.cu"] == {"kv_apply", "kv_fresh"} and found["rope.cu"] == {"rope_kernel"}
