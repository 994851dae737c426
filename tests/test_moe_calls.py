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


# ------------------------------------------------------------------ what the tensors hold

class Fake:
    """A tensor of the current device, as the binding sees it: enough of one for it to be refused."""

    def __init__(self, dtype, shape=(), bits=32):
        self.dtype, self.shape, self.bits, self.device = dtype, shape, bits, "cuda:0"

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE

    def element_size(self):
        return self.bits // 8

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n


CALLS = {"dsv4_add_rms_norm": ("x", "residual", "weight", "res_out", "y", "yq", "yscale"),
         "dsv4_route_experts": ("logits", "bias", "ids", "weights"),
         "dsv4_expert_mlp": ("x", "x_scale", "ids", "weights", "w13", "w2", "out", "workspace")}


def refused(abi, fn, p, **over):
    """The call with raw addresses but for `over`."""
    a = {n: FAKE * (i + 1) for i, n in enumerate(CALLS[fn])}
    if "x_scale" in a:
        a["x_scale"] = None
    a.update(over)
    more = dict(ws_bytes=1) if "workspace" in a else {}
    with pytest.raises(abi.Dsv4Error) as e:
        getattr(abi, fn)(p, *a.values(), stream=0, **more)
    assert e.value.status == ARG, e.value
    return str(e.value)


def test_tensors_of_another_type_are_refused(abi, monkeypatch):
    """A float32 gamma beside 16-bit activations would be read as twice as many wrong channels, 16-bit
    rows where 8-bit ones are said to be, float32 ids: each is named before the library is called."""
    import torch
    monkeypatch.setattr(abi, "_now", lambda: (0, 0))
    bf, f32, half, i32, e4 = torch.bfloat16, torch.float32, torch.float16, torch.int32, torch.float8_e4m3fn
    for dtype, right, wrong in ((abi.BF16, bf, (f32, half, e4, torch.int16)), (abi.F32, f32, (bf, torch.float64, i32))):
        p = _params(abi, dtype=dtype)
        for n in ("x", "residual", "weight", "res_out", "y"):
            for t in wrong:
                m = refused(abi, "dsv4_add_rms_norm", p, **{n: Fake(t, (1 << 20,))})
                assert str(t) in m and str(right) in m
    p = _params(abi)
    for n, t in (("yq", bf), ("yq", torch.float8_e5m2), ("yscale", bf), ("yscale", i32)):
        assert str(t) in refused(abi, "dsv4_add_rms_norm", p, **{n: Fake(t, (1 << 20,))})
    for n, t in (("logits", bf), ("bias", bf), ("bias", i32), ("ids", f32), ("ids", torch.int64), ("weights", i32), ("weights", bf)):
        assert str(t) in refused(abi, "dsv4_route_experts", p, **{n: Fake(t, (1 << 20,))})
    refused(abi, "dsv4_route_experts", _params(abi, logits_dtype=abi.BF16), logits=Fake(f32, (1 << 20,)))
    for n, t in (("x", f32), ("x", e4), ("w13", f32), ("w2", half), ("out", f32), ("ids", f32), ("weights", bf), ("x_scale", bf)):
        assert str(t) in refused(abi, "dsv4_expert_mlp", p, **{n: Fake(t, (1 << 20,))})
    refused(abi, "dsv4_expert_mlp", p, x=Fake(bf, (1 << 20,)), x_scale=Fake(f32, (1 << 20,)))  # 16-bit rows with scales


def test_tensors_of_the_right_type_get_through(abi, monkeypatch):
    """As far as the library, which refuses the sizes (nothing is launched)."""
    import torch
    monkeypatch.setattr(abi, "_now", lambda: (0, 0))
    bf, f32, i32 = (Fake(t, (1 << 20,)) for t in (torch.bfloat16, torch.float32, torch.int32))
    bad = _params(abi, hidden=0, topk=0)
    for e4 in (Fake(torch.float8_e4m3fn, (1 << 20,)), Fake(torch.uint8, (1 << 20,))):
        for call in (lambda: abi.dsv4_add_rms_norm(bad, bf, bf, bf, bf, bf, e4, f32, stream=0),
                     lambda: abi.dsv4_add_rms_norm(_params(abi, hidden=0, dtype=abi.F32), f32, None, f32, None, f32, e4, f32, stream=0),
                     lambda: abi.dsv4_route_experts(bad, f32, f32, i32, f32, stream=0),
                     lambda: abi.dsv4_route_experts(_params(abi, topk=0, logits_dtype=abi.BF16), bf, None, i32, f32, stream=0),
                     lambda: abi.dsv4_expert_mlp(bad, bf, None, i32, f32, bf, bf, bf, f32, ws_bytes=1, stream=0),
                     lambda: abi.dsv4_expert_mlp(bad, e4, f32, i32, f32, bf, bf, bf, e4, ws_bytes=1, stream=0)):
            with pytest.raises(abi.Dsv4Error) as e:
                call()
            assert e.value.status == SHAPE, e.value


def test_tensors_too_small_for_the_call_are_refused(abi, monkeypatch):
    """What the params say is read and written has to be there; more may be."""
    import torch
    monkeypatch.setattr(abi, "_now", lambda: (0, 0))
    bf, f32, i32, e4 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn
    T, h, f, E, k = 5, 272, 48, 16, 2
    p = _params(abi, T=T, hidden=h, inter=f, E=E, topk=k)
    sizes = {"dsv4_add_rms_norm": dict(x=(bf, T * h), residual=(bf, T * h), weight=(bf, h), res_out=(bf, T * h), y=(bf, T * h),
                                       yq=(e4, T * h), yscale=(f32, T * 3)),
             "dsv4_route_experts": dict(logits=(f32, T * E), bias=(f32, E), ids=(i32, T * k), weights=(f32, T * k)),
             "dsv4_expert_mlp": dict(x=(bf, T * h), ids=(i32, T * k), weights=(f32, T * k), w13=(bf, E * 2 * f * h), w2=(bf, E * h * f),
                                     out=(bf, T * h))}
    for fn, args in sizes.items():
        for n, (t, need) in args.items():
            assert str(need) in refused(abi, fn, p, **{n: Fake(t, (need - 1,))})
    refused(abi, "dsv4_expert_mlp", p, x=Fake(e4, (T * h,)), x_scale=Fake(f32, (T * 3 - 1,)))
    full = {fn: {n: Fake(t, (need + 1,)) for n, (t, need) in args.items()} for fn, args in sizes.items()}
    odd = _params(abi, T=T, hidden=h, inter=f, E=E, topk=k, dtype=abi.BF16, eps=-1.0, renorm=2, swiglu_limit=-1.0)
    for fn, args in full.items():  # through to the library, which refuses a flag and launches nothing
        if fn == "dsv4_expert_mlp":
            args = {"x": args.pop("x"), "x_scale": None, **args, "workspace": Fake(torch.uint8, (1,))}
        more = dict(ws_bytes=1) if "workspace" in args else {}
        with pytest.raises(abi.Dsv4Error) as e:
            getattr(abi, fn)(odd, *args.values(), stream=0, **more)
        assert e.value.status == ARG and "null pointer or bad flag" in str(e.value)
    huge = _params(abi, T=2 ** 31 - 1, hidden=2 ** 31 - 1, inter=2 ** 31 - 1, E=2 ** 31 - 1)
    refused(abi, "dsv4_expert_mlp", huge, w13=Fake(bf, (1 << 40,)))


# ------------------------------------------------------------------ the step

@pytest.mark.parametrize("given", ["none", "stream", "handle", "default"])
def test_a_step_is_on_one_stream(abi, monkeypatch, given):
    """The router's product between the calls of the library runs on the stream that they run on."""
    import contextlib

    import torch
    from sparse_long_context_csa_b200 import harness
    now, seen = ["current"], []

    class Stream:
        cuda_stream = 77

    @contextlib.contextmanager
    def on(stream):
        before = now[0]
        if stream is not None:
            now[0] = stream
        yield
        now[0] = before

    def call(*args, stream=None):
        handle = now[0] if stream is None else stream
        seen.append(getattr(handle, "cuda_stream", handle))

    mm = torch.mm
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: type("S", (), {"cuda_stream": handle or "a new one"})())
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: type("S", (), {"cuda_stream": 0})())
    monkeypatch.setattr(torch, "mm", lambda *a, **k: (call(), mm(*a, **k))[1])
    for n in ("dsv4_add_rms_norm", "dsv4_route_experts", "dsv4_expert_mlp"):
        monkeypatch.setattr(abi, n, call)
    p = harness.moe_params(3, 16, 16, 4, 2)
    o = harness.moe_buffers(p, device="cpu")
    x = dict(attn=None, stream=None, gamma=None, router=torch.zeros(4, 16), bias=None, w13=None, w2=None)
    harness.moe_step(p, x, o, **{"none": {}, "stream": dict(stream=Stream()), "handle": dict(stream=77), "default": dict(stream=0)}[given])
    assert seen == [{"none": "current", "default": 0}.get(given, 77)] * 4


# ------------------------------------------------------------------ no tokens

def test_no_tokens_need_no_tensors(abi):
    """A tensor without rows has no address in torch; the sizes and flags are looked at all the same."""
    def nothing(names):
        return {n: None for n in names}

    none = _params(abi, T=0)
    assert _norm(abi, none, **nothing(("x", "residual", "weight", "res_out", "y", "yq", "yscale"))) == OK
    assert _route(abi, none, **nothing(("logits", "bias", "ids", "weights"))) == OK
    assert _experts(abi, none, ws_bytes=0, **nothing(CALLS["dsv4_expert_mlp"])) == OK
    assert _norm(abi, _params(abi, T=0, hidden=0), x=None) == SHAPE
    assert _norm(abi, _params(abi, T=0, eps=-1.0), x=None) == ARG
    assert _route(abi, _params(abi, T=0, topk=0), logits=None) == SHAPE
    assert _route(abi, _params(abi, T=0, renorm=2), logits=None) == ARG
    assert _experts(abi, _params(abi, T=0, inter=0), x=None) == SHAPE
