"""Host-side refusals of dsv4_add_rms_norm, dsv4_route_experts and dsv4_expert_mlp: every call
here returns before any CUDA call, so fake device addresses are never dereferenced."""
import ctypes

import pytest

OK, ARG, SHAPE, ALIGN, DTYPE, WORKSPACE = 0, 1, 2, 3, 4, 7
FAKE = 0x10000


@pytest.fixture(scope="module")
def abi():
    from sparse_long_context_csa_b200 import abi, build
    build.build()
    abi.load()
    return abi


def _params(abi, **kw):
    p = abi.Dsv4MoeParams()
    base = dict(T=4, hidden=256, inter=128, E=16, topk=2, n_group=4, topk_group=2, score_fn=abi.SCORE_SIGMOID, renorm=1,
                scale_pow2=0, dtype=abi.BF16, logits_dtype=abi.F32, eps=1e-6, routed_scale=1.0, swiglu_limit=0.0)
    for k, v in {**base, **kw}.items():
        setattr(p, k, v)
    return p


def _call(abi, fn, p, names, over):
    a = {n: FAKE * (i + 1) for i, n in enumerate(names)}
    a.update(over)
    return getattr(abi.load(), fn)(ctypes.byref(p) if p is not None else None, *a.values(), None)


def _norm(abi, p, **over):
    return _call(abi, "dsv4_add_rms_norm", p, ("x", "residual", "weight", "res_out", "y", "yq", "yscale"), over)


def test_norm_refusals(abi):
    p = _params(abi)
    assert _norm(abi, _params(abi, T=0)) == OK                     # nothing to do, nothing launched
    assert _norm(abi, None) == ARG
    assert _norm(abi, _params(abi, dtype=2)) == DTYPE
    for bad in (dict(T=-1), dict(hidden=0), dict(hidden=(1 << 20) + 1)):
        assert _norm(abi, _params(abi, **bad)) == SHAPE
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(scale_pow2=2)):
        assert _norm(abi, _params(abi, **bad)) == ARG
    for missing in ("x", "weight", "yscale"):
        assert _norm(abi, p, **{missing: None}) == ARG
    assert _norm(abi, p, y=None, yq=None, yscale=None) == ARG      # no output
    assert _norm(abi, p, yq=None) == ARG                           # scales without the 8-bit form
    assert _norm(abi, p, res_out=FAKE, y=FAKE) == ARG              # two outputs in one place
    for n in ("x", "residual", "res_out", "y", "yscale"):           # rows of half the bytes over another's
        assert _norm(abi, p, **{n: FAKE, "yq": FAKE}) == ARG, n
    for n in ("x", "residual", "weight", "res_out", "y", "yq", "yscale"):
        assert _norm(abi, p, **{n: FAKE + 8}) == ALIGN


def _route(abi, p, **over):
    return _call(abi, "dsv4_route_experts", p, ("logits", "bias", "ids", "weights"), over)


def test_route_refusals(abi):
    p = _params(abi)
    assert _route(abi, _params(abi, T=0)) == OK
    assert _route(abi, None) == ARG
    assert _route(abi, _params(abi, logits_dtype=3)) == DTYPE
    for bad in (dict(T=-1), dict(E=0), dict(E=1025, n_group=1), dict(topk=0), dict(topk=33, E=64), dict(n_group=0),
                dict(n_group=3), dict(n_group=64, E=64), dict(topk_group=0), dict(topk_group=5), dict(topk=9)):
        assert _route(abi, _params(abi, **bad)) == SHAPE, bad
    for bad in (dict(score_fn=3), dict(score_fn=-1), dict(renorm=2), dict(routed_scale=float("nan"))):
        assert _route(abi, _params(abi, **bad)) == ARG, bad
    for missing in ("logits", "ids", "weights"):
        assert _route(abi, p, **{missing: None}) == ARG
    for n in ("logits", "bias", "ids", "weights"):
        assert _route(abi, p, **{n: FAKE + 4}) == ALIGN


def _experts(abi, p, ws_bytes=1 << 40, **over):
    names = ("x", "x_scale", "ids", "weights", "w13", "w2", "out", "workspace")
    a = {n: FAKE * (i + 1) for i, n in enumerate(names)}
    a.update(over)
    return abi.load().dsv4_expert_mlp(ctypes.byref(p) if p is not None else None, *a.values(), ws_bytes, None)


def test_experts_refusals(abi):
    p = _params(abi)
    assert _experts(abi, _params(abi, T=0)) == OK
    assert _experts(abi, None) == ARG
    assert _experts(abi, _params(abi, dtype=9)) == DTYPE
    assert _experts(abi, _params(abi, dtype=abi.F32)) == SHAPE     # bf16 operands only
    for bad in (dict(T=-1), dict(hidden=8), dict(hidden=264), dict(inter=0), dict(inter=72), dict(E=0), dict(E=1025),
                dict(topk=0), dict(topk=65), dict(T=1 << 30, topk=2), dict(hidden=(1 << 20) + 16)):
        assert _experts(abi, _params(abi, **bad)) == SHAPE, bad
        assert abi.dsv4_expert_mlp_workspace_bytes(_params(abi, **bad)) == 0
    for bad in (dict(swiglu_limit=-1.0), dict(swiglu_limit=float("nan"))):
        assert _experts(abi, _params(abi, **bad)) == ARG
    for missing in ("x", "ids", "weights", "w13", "w2", "out"):
        assert _experts(abi, p, **{missing: None}) == ARG
    assert _experts(abi, p, out=FAKE) == ARG                       # out over x
    for n in ("x", "x_scale", "ids", "weights", "w13", "w2", "out", "workspace"):
        assert _experts(abi, p, **{n: FAKE + 8}) == ALIGN
    need = abi.dsv4_expert_mlp_workspace_bytes(p)
    assert need > 0
    assert _experts(abi, p, workspace=None) == WORKSPACE
    assert _experts(abi, p, ws_bytes=need - 1) == WORKSPACE


def test_workspace_grows_with_the_rows(abi):
    sizes = [abi.dsv4_expert_mlp_workspace_bytes(_params(abi, T=t, topk=k)) for t, k in ((1, 1), (1, 2), (64, 2), (4096, 8))]
    assert sizes == sorted(sizes) and sizes[0] > 0
    big = abi.dsv4_expert_mlp_workspace_bytes(_params(abi, T=1 << 20, topk=8, hidden=4096, inter=2048))
    assert big > 8 * (1 << 20) * 4096 * 2                          # sizes past 32 bits


def test_binding_raises_with_the_status(abi):
    with pytest.raises(abi.Dsv4Error) as e:
        abi.dsv4_route_experts(_params(abi, topk=0), FAKE, None, FAKE, FAKE, stream=0)
    assert e.value.status == SHAPE


def test_binding_refuses_tensors_that_the_kernels_cannot_read(abi, monkeypatch):
    """A tensor of the host or of another device than the current one, and a strided view, before
    the library is called."""
    import torch
    host = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(abi.Dsv4Error) as e:
        abi.dsv4_add_rms_norm(_params(abi), host, None, FAKE, None, FAKE, stream=0)
    assert e.value.status == ARG and "cpu" in str(e.value)

    class Strided:                                                # a device tensor's view, as the binding sees it
        device = "cuda:0"

        def get_device(self):
            return 0

        def is_contiguous(self):
            return False

        def stride(self):
            return (512, 2)

    monkeypatch.setattr(abi, "_now", lambda: (0, 0))
    with pytest.raises(abi.Dsv4Error) as e:
        abi.dsv4_route_experts(_params(abi), Strided(), None, FAKE, FAKE, stream=0)
    assert e.value.status == ARG and "contiguous" in str(e.value)
    with pytest.raises(abi.Dsv4Error):
        abi.dsv4_expert_mlp(_params(abi), FAKE, None, Strided(), FAKE, FAKE, FAKE, FAKE, FAKE, ws_bytes=1, stream=0)
    monkeypatch.setattr(abi, "_now", lambda: (1, 0))
    with pytest.raises(abi.Dsv4Error) as e:                       # on cuda:0 while cuda:1 is current
        abi.dsv4_route_experts(_params(abi), Strided(), None, FAKE, FAKE, stream=0)
    assert e.value.status == ARG and "current" in str(e.value)


@pytest.mark.parametrize("size", [2, 8])
def test_binding_refuses_ids_and_weights_that_are_not_of_32_bits(abi, monkeypatch, size):
    """What torch.topk returns: of int64 ids, read as 32 bits, every other one would be 0."""
    class Choice:
        device, dtype = "cuda:0", f"{8 * size} bits"

        def get_device(self):
            return 0

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return FAKE

        def element_size(self):
            return size

    monkeypatch.setattr(abi, "_now", lambda: (0, 0))
    for ids, weights in ((Choice(), FAKE), (FAKE, Choice())):
        for call in (lambda: abi.dsv4_route_experts(_params(abi), FAKE, None, ids, weights, stream=0),
                     lambda: abi.dsv4_expert_mlp(_params(abi), FAKE, None, ids, weights, FAKE, FAKE, FAKE, FAKE, ws_bytes=1,
                                                 stream=0)):
            with pytest.raises(abi.Dsv4Error) as e:
                call()
            assert e.value.status == ARG and f"{8 * size} bits" in str(e.value)


def test_calls_without_ctypes(abi):
    """What the callables pass on to the functions that say what is wrong, and what they refuse."""
    import torch
    from sparse_long_context_csa_b200 import _binding
    abi.load()
    p, t = _params(abi), torch.zeros(4, dtype=torch.int32)
    assert abi._route(p, FAKE, None, FAKE, FAKE) is None                # raw pointers
    assert abi._route(p, t, None, t, t) is None                         # not on a GPU
    assert abi._route(p, None, None, None, None) is None
    assert abi._route(p, t, None, t) is None and abi._route() is None   # arguments are missing
    for bad in ((0, 4, 0, 0), (FAKE, 3, 0, 0), (FAKE, 9, 0, 0), (FAKE, 8, 0, 0), (FAKE, 4, 0, 1)):
        with pytest.raises(ValueError):
            _binding.entry(*bad)
