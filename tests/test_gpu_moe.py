"""GPU-vs-oracle parity of dsv4_add_rms_norm, dsv4_route_experts and dsv4_expert_mlp, through the
C ABI binding, against the fp64 oracle (oracle/moe_oracle.py).

Tolerances, from the arithmetic (u = 2^-24, the half step of fp32; bf16 half step 2^-8 and e4m3
half step 2^-4 relative to the value, 2^-10 of the scale below the smallest normal number):

  norm     r is one rounded addition.  The sum of squares has chains of at most hidden/32 + 16
           additions, each square one rounding more and two from r, and enters y through a square
           root: |dy| <= |y| u (0.5 (hidden/32 + 20) + 8), the 8 for the division by hidden, eps,
           the reciprocal square root (2 ulp = 4 u) and two products.  Then the storage's half step.
  scales   max|y| / 448 has y's relative error and one division; a power of two lies in
           [s, 2s] of it.  |q s - y| <= 2^-4 |y| + 2^-10 s + |dy| (+ the division's u).
  weights  exp, log1p and the divisions are within 4 u each; the softmax's argument l - max is
           rounded (relative error u |l - max| of exp), its sum has chains of E/32 + 16: relative
           error u (40 + 2 max|l| + E/32), twice that where the weights are renormalised.
  experts  g and u: K + 2 roundings of sum |w x| (and 2^-8 of each |x| where it is dequantised to
           bf16 inexactly).  silu is 1.1-Lipschitz and a clamp 1-Lipschitz, so with
           |silu(g)| <= |g|: |dh| <= 1.1 |u| dg + |silu g| du + 1.1 dg du + 12 u |h| + 2^-8 |h| (the
           12 for exp, the division and two products), then inter + 2 roundings of sum |w2 h|,
           topk + 2 of the weighted sum, and the output's half step.
"""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu

U, BF, E4 = 2.0 ** -24, 2.0 ** -8, 2.0 ** -4
FN = {"softmax": 0, "sigmoid": 1, "sqrt_softplus": 2}


@pytest.fixture(scope="module")
def abi():
    from sparse_long_context_csa_b200 import abi
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    abi.load()
    return abi


def params(abi, **kw):
    p = abi.Dsv4MoeParams()
    base = dict(T=0, hidden=0, inter=0, E=0, topk=0, n_group=1, topk_group=1, score_fn=0, renorm=0, scale_pow2=0,
                dtype=abi.BF16, logits_dtype=abi.F32, eps=1e-6, routed_scale=1.0, swiglu_limit=0.0)
    for k, v in {**base, **kw}.items():
        setattr(p, k, v)
    return p


def f64(t):
    return t.double().cpu().numpy()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------ norm

def norm_delta(hidden):
    return U * (0.5 * (hidden / 32 + 20) + 8)


def check_norm(x, residual, weight, eps, res_out, y, q, s, pow2):
    bf = x.dtype == torch.bfloat16
    r_ref, y_ref = O.rms_norm(f64(x), None if residual is None else f64(residual), f64(weight), eps)
    half, d = (BF if bf else U), norm_delta(x.shape[1])
    if res_out is not None:
        assert np.all(np.abs(f64(res_out) - r_ref) <= (half + 2 * U) * np.abs(r_ref))
    if y is not None:
        assert np.all(np.abs(f64(y) - y_ref) <= (half + d * (1 + half)) * np.abs(y_ref) + 1e-38)
    if q is None:
        return
    s_ref, s_got = O.group_scales(y_ref), f64(s)
    if pow2:
        assert np.all(np.log2(s_got) == np.round(np.log2(s_got)))
        live = np.abs(y_ref).max() > 0
        assert not live or (np.all(s_got >= s_ref * (1 - 2 * d - 4 * U)) and np.all(s_got <= 2 * s_ref * (1 + 2 * d)))
    else:
        assert np.all(np.abs(s_got - s_ref) <= s_ref * (d + 4 * U))
    wide = np.repeat(s_got, 128, axis=1)[:, :x.shape[1]]
    got = f64(q.float()) * wide
    assert np.all(np.abs(got - y_ref) <= (E4 * (1 + d) + d + 4 * U) * np.abs(y_ref) + 2.0 ** -10 * wide * (1 + d))


NORM_SHAPES = [(1, 4096), (3, 1), (5, 7), (2, 31), (4, 128), (7, 129), (9, 1111), (2, 640), (33, 2048), (17, 8192), (130, 512),
               (2, 8200), (1, 16384), (3, 20001), (1000, 72), (21, 333), (9, 700), (5, 2047), (6, 2049), (600, 256), (3, 32768),
               (2, 40000), (2500, 1111), (10000, 37), (700, 5001), (400, 8191)]                 # more rows than are held at once


@pytest.mark.parametrize("T,hidden", NORM_SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm(abi, T, hidden, dtype):
    for variant, (res, want_y, want_q, pow2) in enumerate([(True, True, False, 0), (True, True, True, 0), (False, False, True, 1),
                                                           (False, True, False, 0), (True, False, True, 1)]):
        g = gen(100 * T + hidden + variant)
        x = (3 * torch.randn(T, hidden, generator=g, device="cuda")).to(dtype)
        residual = torch.randn(T, hidden, generator=g, device="cuda").to(dtype) if res else None
        weight = (1 + 0.3 * torch.randn(hidden, generator=g, device="cuda")).to(dtype)
        p = params(abi, T=T, hidden=hidden, scale_pow2=pow2, dtype=abi.BF16 if dtype == torch.bfloat16 else abi.F32, eps=1e-5)
        guard = 3  # rows behind the last one stay as they were
        new = lambda dt, *sh: torch.full((T + guard, *sh), 5, device="cuda").to(dt)  # noqa: E731
        res_out, y = (new(dtype, hidden) if res else None), (new(dtype, hidden) if want_y else None)
        q = new(torch.float8_e4m3fn, hidden) if want_q else None
        s = new(torch.float32, -(-hidden // 128)) if want_q else None
        abi.dsv4_add_rms_norm(p, x, residual, weight, res_out, y, q, s)
        torch.cuda.synchronize()
        for t in (res_out, y, q, s):
            assert t is None or bool((t[T:].float() == 5).all())
        cut = [None if t is None else t[:T] for t in (res_out, y, q, s)]
        check_norm(x, residual, weight, 1e-5, *cut, pow2)


@pytest.mark.parametrize("T,hidden,dtype", [(5, 4096, torch.bfloat16), (6, 129, torch.float32), (3, 8200, torch.bfloat16),
                                            (9, 333, torch.bfloat16), (3, 5001, torch.bfloat16), (2, 40000, torch.bfloat16),
                                            (3, 1999, torch.float32), (1200, 1111, torch.bfloat16), (9000, 99, torch.float32)])
def test_norm_in_place(abi, T, hidden, dtype):
    """The residual stream updated where it lies, and y written over x."""
    g = gen(9)
    x, residual = (torch.randn(T, hidden, generator=g, device="cuda").to(dtype) for _ in range(2))
    weight = torch.rand(hidden, generator=g, device="cuda").to(dtype)
    x0, r0 = x.clone(), residual.clone()
    p = params(abi, T=T, hidden=hidden, dtype=abi.BF16 if dtype == torch.bfloat16 else abi.F32, eps=1e-6)
    abi.dsv4_add_rms_norm(p, x, residual, weight, residual, x)
    check_norm(x0, r0, weight, 1e-6, residual, x, None, None, 0)


def test_norm_zero_rows_groups_and_non_finite(abi):
    T, hidden = 6, 384
    x = torch.randn(T, hidden, generator=gen(3), device="cuda")
    x[0] = 0                       # an empty row (padding): zeros, scales of 1
    x[1, 128:256] = 0              # an all-zero group
    x[2, 5] = float("nan")         # the row becomes NaN, the others do not
    x[3, 7] = float("inf")
    x[4] *= 1e-30                  # eps decides
    for dt in (torch.float32, torch.bfloat16):
        xi, w = x.to(dt), torch.ones(hidden, device="cuda").to(dt)
        y, q, s = torch.empty_like(xi), torch.empty(T, hidden, device="cuda").to(torch.float8_e4m3fn), torch.empty(T, 3, device="cuda")
        abi.dsv4_add_rms_norm(params(abi, T=T, hidden=hidden, dtype=abi.F32 if dt == torch.float32 else abi.BF16), xi, None, w,
                              None, y, q, s)
        assert bool((y[0] == 0).all()) and bool((s[0] == 1).all()) and bool((q[0].float() == 0).all())
        assert float(s[1, 1]) == 1 and bool((q[1, 128:256].float() == 0).all())
        assert bool(y[2].isnan().all()) and bool(q[2].float().isnan().all())
        assert bool(y[3, 7].isnan()) and bool((y[3, torch.arange(hidden, device="cuda") != 7] == 0).all())
        keep = [1, 4, 5]
        check_norm(xi[keep], None, w, 1e-6, None, y[keep], q[keep], s[keep], 0)


# ------------------------------------------------------------------ routing

def check_route(abi, logits, bias, fn, topk, n_group=1, topk_group=1, renorm=1, scale=2.5):
    T, E = logits.shape
    p = params(abi, T=T, E=E, topk=topk, n_group=n_group, topk_group=topk_group, score_fn=FN[fn], renorm=renorm, routed_scale=scale,
               logits_dtype=abi.F32 if logits.dtype == torch.float32 else abi.BF16)
    ids = torch.full((T + 2, topk), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T + 2, topk), -9.0, device="cuda")
    abi.dsv4_route_experts(p, logits, bias, ids, w)
    torch.cuda.synchronize()
    assert bool((ids[T:] == -9).all()) and bool((w[T:] == -9).all())
    l = f64(logits)
    ref_ids, ref_w = O.route(l, None if bias is None else f64(bias), fn=fn, topk=topk, n_group=n_group, topk_group=topk_group,
                             renorm=bool(renorm), routed_scale=scale)
    np.testing.assert_array_equal(ids[:T].cpu().numpy(), ref_ids)
    finite = l[np.isfinite(l)]
    rel = U * (40 + 2 * (np.abs(finite).max() if finite.size else 0) + E / 32) * (2 if renorm else 1)
    got = f64(w[:T])
    bad = np.isnan(ref_w)
    assert np.array_equal(bad, np.isnan(got))
    assert np.all(np.abs(got - ref_w)[~bad] <= rel * np.abs(ref_w[~bad]) + 1e-37)


ROUTES = [  # T, E, topk, n_group, topk_group
    (1, 1, 1, 1, 1), (3, 2, 2, 1, 1), (65, 8, 3, 1, 1), (64, 256, 6, 1, 1), (129, 256, 8, 8, 4), (33, 60, 4, 1, 1),
    (50, 96, 5, 3, 2), (12, 1023, 8, 3, 2), (5000, 64, 6, 8, 3), (31, 512, 12, 8, 3), (17, 1024, 32, 32, 32), (9, 33, 32, 1, 1), (20, 32, 4, 32, 7), (40, 14, 7, 2, 1),
    (700, 400, 10, 1, 1), (77, 128, 6, 4, 2), (19, 256, 32, 32, 4), (21, 288, 18, 32, 2), (13, 620, 20, 31, 1),
    (9, 512, 32, 16, 1)]                                       # every expert of the groups that stay


@pytest.mark.parametrize("fn", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("T,E,topk,n_group,topk_group", ROUTES)
def test_route(abi, T, E, topk, n_group, topk_group, fn):
    for k, (dt, biased, renorm) in enumerate([(torch.float32, True, 1), (torch.float32, False, 0), (torch.bfloat16, True, 0),
                                              (torch.bfloat16, False, 1)]):
        g = gen(31 * T + E + k)
        logits = (2 * torch.randn(T, E, generator=g, device="cuda")).to(dt)
        bias = 0.2 * torch.randn(E, generator=g, device="cuda") if biased else None
        check_route(abi, logits, bias, fn, topk, n_group, topk_group, renorm)


@pytest.mark.parametrize("fn", ["softmax", "sigmoid", "sqrt_softplus"])
def test_route_ties(abi, fn):
    """Equal logits, few distinct values, with and without groups: the lower index first."""
    g = gen(5)
    few = torch.randint(-2, 3, (200, 64), generator=g, device="cuda").float()
    few[0] = 0
    for bias in (None, torch.zeros(64, device="cuda"), torch.randint(0, 2, (64,), generator=g, device="cuda") * 0.5):
        check_route(abi, few, bias, fn, 7)
        check_route(abi, few, bias, fn, 7, 8, 3)
        check_route(abi, few.bfloat16(), bias, fn, 7, 4, 2)


@pytest.mark.parametrize("fn", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_near_ties(abi, fn, biased):
    """Scores that 32 bits cannot tell apart: saturated sigmoids, neighbouring floats, and biases that
    make up for the difference of the scores to the last bits."""
    T, E = 300, 128
    g = gen(6)
    base = 1 + torch.rand(T, 1, generator=g, device="cuda")
    ulps = torch.randint(0, 40, (T, E), generator=g, device="cuda")
    logits = base * (1 + ulps * 2.0 ** -23)
    logits[100:200] += 20 if fn != "softmax" else 0          # sigmoid is 1 in 32 bits there
    bias = None
    if biased:
        s = torch.from_numpy(np.stack([O.score(fn, r) for r in f64(logits[:1])])).cuda()[0]
        bias = (s.max() - s + 0.25).float()
        logits[1:50] = logits[0]
    check_route(abi, logits, bias, fn, 9)
    check_route(abi, logits, bias, fn, 9, 4, 2)


def test_route_masked_and_non_finite(abi):
    """Logits of -inf and of the lowest value; a row with nothing left; a NaN is chosen last."""
    T, E = 8, 40
    inf = float("inf")
    logits = torch.randn(T, E, generator=gen(8), device="cuda")
    logits[0] = -inf
    logits[1, 3:] = -inf                                       # fewer left than topk
    logits[2] = torch.finfo(torch.float32).min
    logits[3, ::2] = torch.finfo(torch.float32).min
    for fn in ("softmax", "sigmoid", "sqrt_softplus"):
        for renorm in (0, 1):
            check_route(abi, logits, None, fn, 6, renorm=renorm)
            check_route(abi, logits, 0.1 * torch.randn(E, generator=gen(9), device="cuda"), fn, 6, 4, 2, renorm)
    nan = logits.clone()
    nan[4, 1] = float("nan")
    nan[5] = float("nan")
    for fn in ("sigmoid", "sqrt_softplus"):
        check_route(abi, nan, None, fn, 5, renorm=0)
        check_route(abi, nan, 0.1 * torch.randn(E, generator=gen(9), device="cuda"), fn, 5, 4, 2, 0)
    # an expert that everyone has to take does not blur the choice among the others: two experts of
    # equal biases and neighbouring logits in groups of their own
    must = torch.zeros(E, device="cuda")
    must[0] = inf
    close = logits[6:7].repeat(64, 1)
    close[:, 10:] *= 0.01
    close[:, 10], close[:, 11], close[:, 20], close[:, 21] = 3.0, 2.0, 3.0, 2.0
    close[:, 20] += 2.0 ** -21 * (torch.arange(64, device="cuda") % 5 - 2)
    check_route(abi, close, must, "sigmoid", 3, 4, 2, 0)
    # a bias of -inf takes an expert out
    bias = torch.zeros(E, device="cuda")
    bias[:35] = -inf
    check_route(abi, logits, bias, "sigmoid", 5)


@pytest.mark.parametrize("fn", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 3)])
def test_route_neighbours_of_small_scores(abi, fn, groups, kept):
    """Scores of about e^-30, where exp's argument rounds away as much as neighbouring logits differ."""
    T, E = 64, 128
    g = gen(21)
    steps = torch.stack([torch.randperm(E, generator=g, device="cuda") for _ in range(T)])
    logits = -30.0 - 2.0 ** -19 * steps                         # neighbours in fp32
    bias = torch.zeros(E, device="cuda")
    if fn == "softmax":
        logits[:, 5], bias[5] = 0.0, -float("inf")             # nearly all of the sum, not to be chosen
    check_route(abi, logits, bias, fn, 6, groups, kept, 0)
    check_route(abi, logits, None, fn, 6, groups, kept, 0)


# ------------------------------------------------------------------ experts

def experts_inputs(T, hidden, inter, E, topk, seed, x8=None, spread=1.0):
    g = gen(seed)
    x = torch.randn(T, hidden, generator=g, device="cuda").bfloat16()
    scale = None
    if x8 is not None:
        n = -(-hidden // 128)
        scale = torch.rand(T, n, generator=g, device="cuda") * 0.01 + 0.001
        if x8 == "pow2":
            scale = torch.exp2(torch.floor(torch.log2(scale)))
        x = (200 * torch.randn(T, hidden, generator=g, device="cuda")).clamp(-448, 448).to(torch.float8_e4m3fn)
    want = torch.randn(T, E, generator=g, device="cuda") + spread * torch.randn(E, generator=g, device="cuda")
    ids = want.topk(min(topk, E), dim=1).indices.int()
    if topk > E:
        ids = torch.randint(0, E, (T, topk), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand(T, topk, generator=g, device="cuda") + 0.1
    w13 = (torch.randn(E, 2 * inter, hidden, generator=g, device="cuda") * 1.5 / hidden ** 0.5).bfloat16()
    w2 = (torch.randn(E, hidden, inter, generator=g, device="cuda") / inter ** 0.5).bfloat16()
    return x, scale, ids, w, w13, w2


def experts_reference(x, scale, ids, w, w13, w2, limit, inexact, rounded=True):
    """The formula in 64 bits over (token, choice) pairs, one expert at a time, and the error
    bound of the module docstring (torch on the GPU: the oracle's loop over tokens is compared
    with it below)."""
    T, hidden = x.shape
    E, f = w13.shape[0], w13.shape[1] // 2
    xd = x.double()
    if scale is not None:
        xd = xd * scale.double().repeat_interleave(128, 1)[:, :hidden]
    out, tol = torch.zeros_like(xd), torch.zeros_like(xd)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        a, wt = w13[e].double(), w[t, j].double()[:, None]
        p = xd[t] @ a.T
        dp = ((hidden + 2) * U + (BF if inexact else 0)) * (xd[t].abs() @ a.abs().T)
        g, u, dg, du = p[:, :f], p[:, f:], dp[:, :f], dp[:, f:]
        if limit > 0:
            g, u = g.clamp(max=limit), u.clamp(-limit, limit)
        silu = g * torch.sigmoid(g)
        h = silu * u
        dh = 1.1 * u.abs() * dg + silu.abs() * du + 1.1 * dg * du + (12 * U + (BF if rounded else 0)) * h.abs()
        b = w2[e].double()
        y = h @ b.T
        dy = dh @ b.abs().T + (f + 2) * U * ((h.abs() + dh) @ b.abs().T)
        out.index_add_(0, t, wt * y)
        tol.index_add_(0, t, wt.abs() * (dy + (ids.shape[1] + 2) * U * (y.abs() + dy)))
    return out, tol + BF * (out.abs() + tol) + 1e-30


def run_experts(abi, ins, limit=0.0, out=None, ws=None, stream=None):
    x, scale, ids, w, w13, w2 = ins
    T, hidden = x.shape
    p = params(abi, T=T, hidden=hidden, inter=w13.shape[1] // 2, E=w13.shape[0], topk=ids.shape[1], swiglu_limit=limit)
    if out is None:
        out = torch.full((T + 3, hidden), 5.0, device="cuda", dtype=torch.bfloat16)
    if ws is None:  # what it holds before the call does not matter: NaN patterns
        ws = torch.full((abi.dsv4_expert_mlp_workspace_bytes(p),), 255, dtype=torch.uint8, device="cuda")
    abi.dsv4_expert_mlp(p, x, scale, ids, w, w13, w2, out, ws, stream=stream)
    return out


def check_experts(abi, ins, limit=0.0, inexact=False):
    T = ins[0].shape[0]
    out = run_experts(abi, ins, limit)
    abi.dsv4_device_check()
    assert bool((out[T:] == 5).all())
    few = T <= 3 and ins[2].numel() <= 32 and max(ins[4].shape[2], ins[5].shape[2]) <= 8192  # h stays in 32 bits
    ref, tol = experts_reference(*ins, limit, inexact, not few)
    err = (out[:T].double() - ref).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol).max()):.2f} of the bound"
    return out[:T], ref


EXPERTS = [  # T, hidden, inter, E, topk
    (1, 16, 16, 1, 1), (1, 256, 128, 8, 2), (1, 4096, 2048, 8, 6), (2, 144, 80, 5, 3), (3, 1040, 272, 16, 4), (5, 512, 256, 64, 6),
    (8, 2048, 512, 4, 2), (17, 128, 1040, 3, 2), (31, 272, 48, 128, 8), (64, 1024, 512, 16, 4), (65, 96, 112, 2, 1),
    (100, 640, 384, 1, 1), (129, 512, 144, 7, 3), (257, 384, 256, 4, 2), (300, 1024, 768, 64, 6), (777, 256, 128, 1000, 5),
    (1000, 528, 304, 8, 4), (2049, 512, 512, 16, 2),
    (2, 4112, 4112, 3, 2), (3, 8192, 272, 4, 3), (1, 8208, 64, 3, 2), (2, 64, 8208, 3, 2),  # widths at the few-token path's ends
    (3, 512, 256, 2, 2), (4, 512, 256, 2, 2), (3, 16, 16, 2, 11), (1, 48, 16, 40, 33),      # tokens and pairs at its ends
    (272, 256, 128, 1, 1), (511, 128, 64, 1, 1), (600, 192, 80, 511, 7), (600, 192, 80, 512, 7), (1025, 128, 32, 1, 4),
    (512, 64, 16, 9, 1), (513, 64, 16, 9, 1), (256, 2064, 32, 1000, 2), (128, 4112, 16, 2, 4),  # pairs put in order by the gather or before it
    (1030, 2064, 32, 4, 3), (2050, 2064, 16, 3, 2), (4100, 4112, 16, 2, 2)]                 # rows wider than a CTA, and than L2 keeps


@pytest.mark.parametrize("T,hidden,inter,E,topk", EXPERTS)
def test_experts(abi, T, hidden, inter, E, topk):
    check_experts(abi, experts_inputs(T, hidden, inter, E, topk, T + hidden), limit=0.0)
    check_experts(abi, experts_inputs(T, hidden, inter, E, topk, T + hidden + 1), limit=1.25)


@pytest.mark.parametrize("T,hidden,inter,E,topk", [(1, 256, 128, 8, 2), (6, 1040, 64, 4, 2), (70, 384, 256, 8, 3), (600, 528, 128, 4, 2)])
@pytest.mark.parametrize("x8", ["pow2", "any"])
def test_experts_of_8_bit_rows(abi, T, hidden, inter, E, topk, x8):
    check_experts(abi, experts_inputs(T, hidden, inter, E, topk, 7, x8=x8), limit=10.0, inexact=x8 == "any")


@pytest.mark.parametrize("T", [1, 4, 40, 500])
def test_experts_formula_is_the_oracles(abi, T):
    """The reference above against the oracle's loop over tokens, on a few of the tokens."""
    ins = experts_inputs(T, 128, 64, 6, 3, 77)
    ref, _ = experts_reference(*ins, 2.0, False)
    rows = sorted({0, T // 2, T - 1})
    x, _, ids, w, w13, w2 = ins
    want = O.expert_mlp(f64(x)[rows], ids.cpu().numpy()[rows], f64(w)[rows], f64(w13), f64(w2), 2.0)
    assert np.allclose(f64(ref)[rows], want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("T", [1, 3, 8, 40, 700])
def test_experts_dropped_repeated_and_skewed(abi, T):
    ins = list(experts_inputs(T, 256, 144, 9, 4, 21))
    ids = ins[2]
    # every token asks one expert
    ins[2] = torch.full_like(ids, 4)
    check_experts(abi, ins)
    # ids outside the experts contribute nothing, whatever their weight; a token with none is zero
    bad = ids.clone()
    bad[:, 1], bad[T // 2], bad[-1, 0] = -1, 9, 2 ** 31 - 1
    bad[0, 2] = -2 ** 31
    ins[2] = bad
    ins[3] = ins[3].clone()
    ins[3][:, 1] = float("nan")
    safe = list(ins)
    safe[3] = torch.where((bad >= 0) & (bad < 9), ins[3], torch.zeros_like(ins[3]))
    out = run_experts(abi, ins)
    ref, tol = experts_reference(*safe, 0.0, False)
    assert bool(((out[:T].double() - ref).abs() <= tol).all()) and bool((out[T // 2] == 0).all())
    # the same expert twice in a row
    two = ids.clone()
    two[:, 1] = two[:, 0]
    ins[2], ins[3] = two, safe[3] + 0.5
    check_experts(abi, ins)
    # nothing at all
    ins[2] = torch.full_like(ids, -1)
    out = run_experts(abi, ins)
    assert bool((out[:T] == 0).all())


def test_experts_non_finite_rows_stay_with_their_token(abi):
    """A NaN in one token's row (padding that was never written) reaches no other token."""
    for T in (4, 90, 400):
        ins = list(experts_inputs(T, 256, 128, 4, 2, 5))
        ins[0] = ins[0].clone()
        ins[0][T // 2] = float("nan")
        ins[0][0, 3] = float("inf")
        out = run_experts(abi, ins)[:T]
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[[0, T // 2]] = False
        ref, tol = experts_reference(*[v[keep] if i in (0, 2, 3) else v for i, v in enumerate(ins)], 0.0, False)
        assert bool(out[T // 2].isnan().all())
        assert bool(((out[keep].double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("T,E,topk", [(1, 8, 2), (6, 8, 4), (48, 16, 4), (900, 8, 2)])
def test_experts_are_the_same_bits_every_time(abi, T, E, topk):
    ins = experts_inputs(T, 512, 256, E, topk, 11)
    first = run_experts(abi, ins).clone()
    for _ in range(4):
        assert torch.equal(run_experts(abi, ins), first)


# ------------------------------------------------------------------ together

@pytest.fixture(scope="module")
def harness(abi):
    from sparse_long_context_csa_b200 import harness
    return harness


def layer_inputs(p, seed):
    g = gen(seed)
    rnd = lambda *sh: torch.randn(sh, generator=g, device="cuda")  # noqa: E731
    return dict(attn=rnd(p.T, p.hidden).bfloat16(), stream=rnd(p.T, p.hidden).bfloat16(), gamma=(1 + 0.1 * rnd(p.hidden)).bfloat16(),
                router=rnd(p.E, p.hidden) / p.hidden ** 0.5, bias=0.1 * rnd(p.E),
                w13=(rnd(p.E, 2 * p.inter, p.hidden) / p.hidden ** 0.5).bfloat16(),
                w2=(rnd(p.E, p.hidden, p.inter) / p.inter ** 0.5).bfloat16())


def layer_params(harness, T, eight_bit):
    return harness.moe_params(T, 512, 256, 16, 4, n_group=4, topk_group=2, routed_scale=1.5, swiglu_limit=7.0, eight_bit=eight_bit)


def check_layer(p, x, o):
    """Each operator against the formula on the inputs that it was given."""
    check_norm(x["attn"], x["stream"], x["gamma"], 1e-6, o["stream"], o["y"], o["q"], o["q_scale"], p.scale_pow2)
    ids, w = O.route(f64(o["logits"]), f64(x["bias"]), fn="sqrt_softplus", topk=p.topk, n_group=4, topk_group=2, renorm=True,
                     routed_scale=1.5)
    np.testing.assert_array_equal(o["ids"].cpu().numpy(), ids)
    assert np.allclose(f64(o["weights"]), w, rtol=1e-5)
    rows, scale = (o["y"], None) if o["q"] is None else (o["q"], o["q_scale"])
    ref, tol = experts_reference(rows, scale, o["ids"], o["weights"], x["w13"], x["w2"], 7.0, False)
    assert bool(((o["out"].double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("eight_bit", [False, True])
@pytest.mark.parametrize("T", [1, 7, 64, 513, 1100])
def test_the_operators_together(abi, harness, T, eight_bit):
    p = layer_params(harness, T, eight_bit)
    x, o = layer_inputs(p, T), harness.moe_buffers(p)
    harness.moe_step(p, x, o)
    check_layer(p, x, o)
    abi.dsv4_device_check()


@pytest.mark.parametrize("T", [1, 5, 130])
def test_captured_and_replayed_on_another_stream(abi, harness, T):
    p = layer_params(harness, T, True)
    x, o = layer_inputs(p, T), harness.moe_buffers(p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        harness.moe_step(p, x, o)                  # warm-up outside the capture
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            harness.moe_step(p, x, o)
    for seed in (1, 2):
        fresh = layer_inputs(p, 100 + seed)
        for n in ("attn", "stream", "bias"):
            x[n].copy_(fresh[n])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
            graph.replay()                         # two in a row share the workspace
        torch.cuda.synchronize()
        check_layer(p, x, o)


def test_two_graphs_share_a_workspace(abi):
    """Calls of other sizes captured into two graphs, replayed in turn over one workspace."""
    ins = [experts_inputs(T, 256, 128, 8, k, T) for T, k in ((90, 2), (2, 4), (2100, 2))]
    want = [run_experts(abi, i).clone() for i in ins]
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    outs = [torch.full_like(w, 5.0) for w in want]
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i, o in zip(ins, outs):
            run_experts(abi, i, out=o, ws=ws)
            side.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                run_experts(abi, i, out=o, ws=ws)
            graphs.append(graph)
        for o in outs:
            o.fill_(5.0)
        for _ in range(3):
            for k in (0, 1, 2, 1, 0):
                graphs[k].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("T", [1, 40])
def test_experts_saturated_gates(abi, T):
    """Gates far below zero (silu underflows) and far above, with and without the clamp."""
    x, _, ids, w, w13, w2 = experts_inputs(T, 128, 64, 4, 2, 3)
    ins = (x, None, ids, w, (60 * w13.float()).bfloat16(), w2)
    check_experts(abi, ins)
    check_experts(abi, ins, limit=10.0)


def test_two_calls_at_once_with_a_workspace_each(abi):
    a, b = (experts_inputs(T, 512, 256, 8, 2, T) for T in (600, 30))
    want = [run_experts(abi, i).clone() for i in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [run_experts(abi, i, out=torch.full_like(w, 5.0), stream=s) for i, w, s in zip((a, b), want, streams)
               if s.wait_stream(torch.cuda.current_stream()) is None]
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("shapes", [[(600, 192, 80, 511, 7), (600, 192, 80, 512, 7)], [(3, 8192, 272, 4, 3), (2, 144, 80, 5, 3)]])
def test_two_threads_at_once(abi, shapes):
    """Calls that need different amounts of shared memory, by threads that do not wait for each other."""
    from concurrent.futures import ThreadPoolExecutor
    ins = [experts_inputs(*s, 40 + i) for i, s in enumerate(shapes)]
    want = [run_experts(abi, i) for i in ins]
    torch.cuda.synchronize()

    def work(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            ws = torch.empty(want[k].numel() * 64 + (1 << 24), dtype=torch.uint8, device="cuda")
            out = [run_experts(abi, ins[k], ws=ws) for _ in range(200)]
            torch.cuda.current_stream().synchronize()
        return out

    with ThreadPoolExecutor(2) as pool:
        for got, w in zip(pool.map(work, range(2)), want):
            assert all(torch.equal(g, w) for g in got)
    abi.dsv4_device_check()


def test_ways_to_call(abi):
    """Tensors on the current stream, a stream that is given, raw pointers: the same results; what is refused."""
    from sparse_long_context_csa_b200 import _binding  # noqa: F401
    T, E, k = 33, 48, 5
    p = params(abi, T=T, E=E, topk=k, score_fn=FN["sigmoid"], renorm=1, routed_scale=1.0, logits_dtype=abi.F32)
    logits = torch.nn.Parameter(torch.randn(T, E, generator=gen(31), device="cuda"))
    bias = torch.randn(E, generator=gen(32), device="cuda")

    def outputs():
        return torch.full((T, k), -9, dtype=torch.int32, device="cuda"), torch.full((T, k), -9.0, device="cuda")

    got = []
    for way in range(4):
        ids, w = outputs()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        if way == 0:
            assert abi._route(p, logits, bias, ids, w) == 0
        elif way == 1:
            abi.dsv4_route_experts(p, logits, bias, ids, w, stream=side)
        elif way == 2:
            abi.dsv4_route_experts(p, logits.data_ptr(), bias.data_ptr(), ids.data_ptr(), w.data_ptr(), stream=side.cuda_stream)
        else:
            with torch.cuda.stream(side):
                assert abi._route(p, logits, bias, ids, w) == 0
                got.append((ids.clone(), w.clone()))
            torch.cuda.current_stream().wait_stream(side)
            continue
        torch.cuda.current_stream().wait_stream(side)
        got.append((ids, w))
    torch.cuda.synchronize()
    assert int(got[0][0].min()) >= 0
    for ids, w in got[1:]:
        assert torch.equal(ids, got[0][0]) and torch.equal(w, got[0][1])
    ids, w = outputs()
    for bad in ((logits.t().contiguous().t(), bias, ids, w), (logits, bias.cpu(), ids, w), (logits, bias, ids.long(), w),
                (logits, bias, ids, w.bfloat16()), (logits, bias.double(), ids, w), (logits.cpu(), bias, ids, w)):
        with pytest.raises(abi.Dsv4Error):
            abi.dsv4_route_experts(p, *bad)
    with pytest.raises(abi.Dsv4Error):
        abi.dsv4_route_experts(p, logits, bias, None, w)
    torch.cuda.synchronize()
    assert int(ids.max()) == -9                                     # a refused call writes nothing


def test_no_tokens(abi):
    e = torch.empty(0, device="cuda")
    p = params(abi, T=0, hidden=128, inter=64, E=4, topk=2)
    z = torch.zeros(16, device="cuda")
    abi.dsv4_add_rms_norm(p, z, None, z, None, z)
    abi.dsv4_route_experts(p, z, None, z, z)
    abi.dsv4_expert_mlp(p, z, None, z, z, z, z, torch.zeros(16, device="cuda"), None)
    assert bool((z == 0).all()) and e.numel() == 0
