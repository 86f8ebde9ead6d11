"""Kernels that are launched while the kernel before them still runs read what it writes by ordinary loads.

The read-only path (__ldg, ld.global.nc, or what a compiler makes of a `const ... __restrict__` parameter) is for memory that
nothing writes during a kernel's life.  An early kernel's life begins before the one in front of it has ended, and its wait
orders ordinary loads only."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "diffusion_transformer_denoiser_gb300", "csrc")
READ_ONLY = re.compile(r"__ldg\s*\(|ld\.global\.nc|ld\.global\.[\w.]*\.nc")


def _kernels(text):
    """(name, parameters, body) of every kernel."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__global__([^{}]*)\{", text):
        head, depth, i = m.group(1).rstrip(), 0, 0
        for i in range(len(head) - 1, -1, -1):  # the parameters are the last parentheses
            depth += {")": 1, "(": -1}.get(head[i], 0)
            if depth == 0:
                break
        depth, end = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
        yield re.search(r"(\w+)\s*$", head[:i]).group(1), head[i + 1:-1], text[m.end():end]


def _early(text):
    return [f for f in _kernels(text) if "grid_dep_wait()" in f[2]]


@pytest.mark.parametrize("name", ["values.cuh", "norm_rows.cuh", "layer_norm.cu", "norm_bwd.cu", "grads.cu"])
def test_no_read_only_loads(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    assert not READ_ONLY.search(re.sub(r"//[^\n]*", "", text))
    for kernel, params, _ in _early(text):
        assert not re.search(r"const[^,]*\*\s*__restrict__", params), kernel


@pytest.mark.parametrize("file,names", [("attention.cu", ["attn_prepare_kernel", "attn_fwd_kernel"]),
                                        ("attention_bwd.cu", ["attn_bwd_rows_kernel", "attn_bwd_kernel"]),
                                        ("elementwise.cu", ["qk_gain_sum_kernel"])])
def test_the_attention_pass(file, names):
    """The attention's output and its log-sum-exp, the output's gradient, the gains' parts: the call before has just written them."""
    with open(os.path.join(CSRC, file)) as f:
        early = {k: (params, body) for k, params, body in _early(f.read())}
    for kernel in names:
        params, body = early[kernel]
        assert not READ_ONLY.search(body), kernel
        assert not re.search(r"const[^,]*\*\s*__restrict__", params), kernel


def test_the_search_finds_them():
    text = """
    __global__ void f(const float* __restrict__ p, float* o) {  // __ldg(
      grid_dep_wait();
      o[0] = p[0];
    }"""
    assert [f[0] for f in _early(text)] == ["f"] and re.search(r"const[^,]*\*\s*__restrict__", _early(text)[0][1])
    assert not READ_ONLY.search("__ldcg(p)") and READ_ONLY.search("__ldg(p)") and READ_ONLY.search("ld.global.nc.v4.u32")
    with open(os.path.join(CSRC, "norm_bwd.cu")) as f:
        assert {k for k, _, _ in _early(f.read())} == {"norm_bwd_kernel", "norm_sum_kernel"}
