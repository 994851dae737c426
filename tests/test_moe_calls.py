"""Host side of dsv4_add_rms_norm, dsv4_route_experts and dsv4_expert_mlp: workspace sizes, what is
refused and what is not, and the build of the binding.  Nothing here launches a kernel."""
import ctypes

import pytest

from test_moe_host import FAKE, abi, _experts, _norm, _params, _route  # noqa: F401

OK, ARG, SHAPE = 0, 1, 2


@pytest.mark.parametrize("hidden,inter,E", [(4096, 4096, 64), (2048, 1408, 32), (4096, 2048, 64), (16, 8192, 8), (16, 8208, 4),
                                            (8208, 16, 1024), (16, 16, 1)])
def test_a_workspace_of_the_largest_call_is_enough(abi, hidden, inter, E):
    """The size never falls with the tokens or the choices: what is sized for the largest batch
    serves every smaller one, through any path."""
    def size(T, k):
        return abi.dsv4_expert_mlp_workspace_bytes(_params(abi, T=T, topk=k, hidden=hidden, inter=inter, E=E))

    tokens = [*range(0, 66), 500, 512, 513, 1024, 2047, 2048, 2049, 4096, 4097, 5000]
    table = [[size(T, k) for T in tokens] for k in range(1, 65)]
    assert table[0][1] > 0
    for row in table:
        assert row == sorted(row)
    for column in zip(*table):
        assert list(column) == sorted(column)


# ------------------------------------------------------------------ the build of the binding

@pytest.fixture
def bare(monkeypatch, tmp_path):
    """The build's module with a binding of its own to build."""
    from sparse_long_context_csa_b200 import build
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    return build


@pytest.mark.parametrize("compiler", ["/nowhere/g++", "false"])
def test_a_compiler_that_fails_leaves_the_library(bare, monkeypatch, tmp_path, compiler):
    """Without a C++ compiler, or without what the binding's source needs, the library is all there is,
    and its calls go through ctypes; a binding of older sources does not stay behind."""
    import os
    monkeypatch.setenv("CXX", compiler)
    (tmp_path / "_binding.so").write_bytes(b"of older sources")
    os.utime(tmp_path / "_binding.so", (1, 1))
    with pytest.warns(UserWarning, match="ctypes"):
        assert bare.build() == bare.LIB
    assert not (tmp_path / "_binding.so").exists()


def test_an_interpreter_without_torch_leaves_the_library(bare, monkeypatch):
    import importlib.util
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    with pytest.warns(UserWarning, match="ctypes"):
        assert bare.build() == bare.LIB


def test_the_binding_is_built_where_it_can_be(bare, tmp_path):
    import warnings
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert bare.build() == bare.LIB
    assert (tmp_path / "_binding.so").exists()
