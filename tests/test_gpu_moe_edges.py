"""The norm, the routing and the experts at the ends of their ranges: against the fp64 oracle
(oracle/moe_oracle.py), with the bounds that tests/test_gpu_moe.py derives where none is given."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from test_gpu_moe import FN, abi, check_route, experts_inputs, f64, gen, params, run_experts  # noqa: F401

pytestmark = pytest.mark.gpu

FNS = ["softmax", "sigmoid", "sqrt_softplus"]


# ------------------------------------------------------------------ groups of negative 16-bit logits

def close_sums(fn, n):
    """n times two pairs of bf16 logits below zero whose scores' sums are closer than a bf16 logit's last
    bits but further than 64 bits can blur: [n, 2, 2], the larger sum first."""
    step = np.arange(128, 256, dtype=np.float64)
    v = -np.concatenate([step * 2.0 ** e for e in (-8, -7, -6, -5)])           # -0.5 .. -8
    s = np.exp(v) if fn == "softmax" else O.score(fn, v)
    i, j = np.triu_indices(len(v), 1)
    total = s[i] + s[j]
    at = np.argsort(total)
    gap = np.diff(total[at]) / total[at][1:]
    some = np.random.default_rng(3).permutation(np.flatnonzero((gap > 2e-8) & (gap < 3e-5)))[:n]
    lo, hi = at[some], at[some + 1]
    return np.stack([np.stack([v[i[hi]], v[j[hi]]], 1), np.stack([v[i[lo]], v[j[lo]]], 1)], 1)


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("E,n_group", [(256, 8), (1024, 8), (60, 4)])
def test_groups_of_negative_16_bit_logits(abi, fn, E, n_group):
    """Without a bias, where the two best of two groups are below zero and their sums nearly equal."""
    T, per = 400, E // n_group
    pairs = close_sums(fn, T)
    assert len(pairs) == T
    rng = np.random.default_rng(E)
    logits = np.full((T, E), -30.0)
    for t in range(T):
        groups = rng.choice(n_group, 2, replace=False)
        for g, two in zip(groups, pairs[t]):
            logits[t, g * per + rng.choice(per, 2, replace=False)] = rng.permutation(two)
    if fn == "sigmoid":
        logits[0] = -30.0
        logits[0, [3, 7]] = -2.984375, -1.6328125
        logits[0, [per + 1, per + 5]] = -2.265625, -2.015625
    x = torch.from_numpy(logits).cuda().bfloat16()
    assert np.array_equal(f64(x), logits)
    check_route(abi, x, None, fn, 3, n_group, 1)


@pytest.mark.parametrize("fn", FNS)
def test_groups_of_many_negative_16_bit_logits(abi, fn):
    T, E, n_group, kept, k = 200_000, 1024, 8, 4, 4
    x = (-6 + torch.randn(T, E, generator=gen(17), device="cuda")).bfloat16()
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    abi.dsv4_route_experts(params(abi, T=T, E=E, topk=k, n_group=n_group, topk_group=kept, score_fn=FN[fn], logits_dtype=abi.BF16), x, None,
                           ids, w)
    for a in range(0, T, 20_000):                       # the formula in 64 bits
        l = x[a:a + 20_000].double()
        s = l.softmax(1) if fn == "softmax" else l.sigmoid() if fn == "sigmoid" else torch.log1p(l.exp()).sqrt()
        two = s.unflatten(1, (n_group, -1)).sort(2, descending=True).values[:, :, :2].sum(2)
        best = two.sort(dim=1, descending=True, stable=True).indices[:, :kept]
        keep = torch.zeros_like(two, dtype=torch.bool).scatter_(1, best, True).repeat_interleave(E // n_group, 1)
        want = torch.where(keep, l, -torch.inf).sort(dim=1, descending=True, stable=True).indices[:, :k]
        wrong = (ids[a:a + 20_000] != want).any(1)
        assert not bool(wrong.any()), f"{int(wrong.sum())} tokens"


# ------------------------------------------------------------------ scores near fp32's lower end

@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("E,topk,n_group,kept", [(64, 6, 1, 1), (256, 8, 8, 4), (1023, 8, 3, 2)])
def test_sqrt_softplus_of_very_negative_logits(abi, E, topk, n_group, kept, renorm):
    """sqrt(log(1 + e^l)) is about e^(l/2): 1e-19 and less, but not nothing beside the 1e-20 of the sum."""
    T = 60
    for k, (dt, bias) in enumerate([(torch.float32, None), (torch.bfloat16, None), (torch.float32, torch.zeros(E, device="cuda")),
                                    (torch.bfloat16, torch.zeros(E, device="cuda"))]):
        l = -85 - 25 * torch.rand(T, E, generator=gen(40 + k + E), device="cuda")
        l[0] = -90.0
        l[1] = torch.linspace(-10, -24, E, device="cuda")              # across the change of the formula
        check_route(abi, l.to(dt), bias, "sqrt_softplus", topk, n_group, kept, renorm)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_sqrt_softplus_groups_of_very_negative_logits(abi, dt, biased):
    """Two scores of e^-43.75 are more than one of e^-43.25."""
    E, n_group, per = 64, 4, 16
    l = torch.full((3, E), -200.0, device="cuda")
    l[:, 0], l[:, per], l[:, per + 1] = -86.5, -87.5, -87.5
    l[1, 0] = -86.0
    l[2, 2 * per:2 * per + 2] = -87.25
    check_route(abi, l.to(dt), torch.zeros(E, device="cuda") if biased else None, "sqrt_softplus", 2, n_group, 1, 0)


# ------------------------------------------------------------------ a softmax of NaN

@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("E,n_group,kept", [(40, 1, 1), (64, 4, 2), (1023, 3, 1)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_softmax_of_nan(abi, dt, E, n_group, kept, renorm):
    """A NaN makes every score of its row NaN, whatever stands beside it; the rows around it stay."""
    inf, nan = float("inf"), float("nan")
    logits = torch.randn(7, E, generator=gen(50), device="cuda")
    logits[1] = nan
    logits[2] = -inf
    logits[2, E // 2] = nan                                       # nothing else but -inf
    logits[3, 1] = nan
    logits[4] = -inf
    logits[5, 2] = inf
    bias = torch.linspace(0, 1, E, device="cuda")
    for b in (None, bias):
        with np.errstate(invalid="ignore"):
            check_route(abi, logits.to(dt), b, "softmax", 5, n_group, kept, renorm)


# ------------------------------------------------------------------ two calls at once

def test_two_calls_at_once_on_streams_of_their_own(abi):
    """Outputs and workspaces are there, filled, before the streams start and until both have ended."""
    calls = [experts_inputs(T, 512, 256, 8, 2, T) for T in (600, 30)]
    want = [run_experts(abi, i).clone() for i in calls]
    sizes = [abi.dsv4_expert_mlp_workspace_bytes(params(abi, T=i[0].shape[0], hidden=512, inter=256, E=8, topk=2)) for i in calls]
    spaces = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    outs = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        for t in spaces:
            t.fill_(255)
        for t in outs:
            t.fill_(5.0)
        torch.cuda.synchronize()
        for i, o, ws, s in zip(calls, outs, spaces, streams):
            run_experts(abi, i, out=o, ws=ws, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    abi.dsv4_device_check()


# ------------------------------------------------------------------ what the tensors hold

def test_tensors_of_another_type_are_refused(abi):
    """By the calls without ctypes, which leave them to the functions that say what is wrong."""
    T, h = 4, 256
    x, w, y = (torch.ones(n, h, device="cuda", dtype=torch.bfloat16) for n in (T, 1, T))
    q, s = torch.empty(T, h, device="cuda", dtype=torch.float8_e4m3fn), torch.empty(T, 2, device="cuda")
    p = params(abi, T=T, hidden=h)
    right = [x, x, w, y.clone(), y, q, s]
    assert abi._norm(p, *right) == 0 and abi._norm(p, *right[:5], q.view(torch.uint8), s) == 0
    for i, wrong in ((0, x.float()), (1, x.float()), (2, w.float()), (2, w.half()), (3, y.float()), (4, y.float()), (5, y), (5, q.view(torch.int8)),
                     (6, s.int()), (6, s.double())):
        args = [*right[:i], wrong, *right[i + 1:]]
        assert abi._norm(p, *args) is None
        with pytest.raises(abi.Dsv4Error) as e:
            abi.dsv4_add_rms_norm(p, *args)
        assert e.value.status == 1 and str(wrong.dtype) in str(e.value)
    ins = experts_inputs(T, 256, 128, 8, 2, 1)
    p = params(abi, T=T, hidden=256, inter=128, E=8, topk=2)
    ws = torch.empty(abi.dsv4_expert_mlp_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    right = [*ins, torch.empty_like(ins[0]), ws]
    assert abi._experts(p, *right) == 0
    x8, scale = experts_inputs(T, 256, 128, 8, 2, 1, x8="pow2")[:2]
    assert abi._experts(p, x8, scale, *right[2:]) == 0
    for over in ({0: x8}, {1: scale}, {0: x8, 1: scale.bfloat16()}, {2: ins[2].float()}, {2: ins[2].long()}, {3: ins[3].int()},
                 {4: ins[4].float()}, {5: ins[5].float()}, {6: torch.empty(T, 256, device="cuda")}):
        args = [over.get(i, t) for i, t in enumerate(right)]
        assert abi._experts(p, *args) is None
        with pytest.raises(abi.Dsv4Error) as e:
            abi.dsv4_expert_mlp(p, *args)
        assert e.value.status == 1
    p = params(abi, T=T, E=8, topk=2, logits_dtype=abi.BF16)
    ids, weights = torch.empty(T, 2, dtype=torch.int32, device="cuda"), torch.empty(T, 2, device="cuda")
    logits = torch.zeros(T, 8, device="cuda")
    assert abi._route(p, logits, None, ids, weights) is None and abi._route(p, logits.bfloat16(), None, ids, weights) == 0
    assert abi._route(p, logits.bfloat16(), None, ids.float(), weights) is None
    torch.cuda.synchronize()


def test_tensors_too_small_for_the_call_are_refused(abi):
    T, h, E, k = 6, 384, 8, 2
    p = params(abi, T=T, hidden=h, inter=128, E=E, topk=k)
    x, w = torch.ones(T, h, device="cuda", dtype=torch.bfloat16), torch.ones(h, device="cuda", dtype=torch.bfloat16)
    q, s = torch.empty(T, h, device="cuda", dtype=torch.float8_e4m3fn), torch.empty(T, 3, device="cuda")
    ids, weights = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.ones(T, k, device="cuda")
    logits, bias = torch.zeros(T, E, device="cuda"), torch.zeros(E, device="cuda")
    w13, w2 = torch.zeros(E, 256, h, device="cuda").bfloat16(), torch.zeros(E, h, 128, device="cuda").bfloat16()
    ws = torch.empty(abi.dsv4_expert_mlp_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    for short, call, args in ((abi._norm, abi.dsv4_add_rms_norm, [x, x.clone(), w, torch.empty_like(x), torch.empty_like(x), q, s]),
                              (abi._route, abi.dsv4_route_experts, [logits, bias, ids, weights]),
                              (abi._experts, abi.dsv4_expert_mlp, [x, None, ids, weights, w13, w2, torch.empty_like(x), ws]),
                              (abi._experts, abi.dsv4_expert_mlp, [q, s, ids, weights, w13, w2, torch.empty_like(x), ws])):
        assert short(p, *args) == 0
        for i, t in enumerate(args):
            if t is None:
                continue
            less = [*args[:i], t.flatten()[:-1], *args[i + 1:]]
            if t is not ws:                          # the library says what is wrong with a workspace
                assert short(p, *less) is None
            with pytest.raises(abi.Dsv4Error) as e:
                call(p, *less)
            assert e.value.status == (7 if t is ws else 1)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ the step

def layer(harness, T, seed=0):
    p = harness.moe_params(T, 512, 256, 16, 4, n_group=4, topk_group=2, routed_scale=1.5, swiglu_limit=7.0)
    g = gen(seed)
    rnd = lambda *sh: torch.randn(sh, generator=g, device="cuda")  # noqa: E731
    return p, dict(attn=rnd(T, 512).bfloat16(), stream=rnd(T, 512).bfloat16(), gamma=(1 + 0.1 * rnd(512)).bfloat16(),
                   router=rnd(16, 512) / 512 ** 0.5, bias=0.1 * rnd(16), w13=(rnd(16, 512, 512) / 512 ** 0.5).bfloat16(),
                   w2=(rnd(16, 512, 256) / 256 ** 0.5).bfloat16())


@pytest.mark.parametrize("T", [1, 700])
def test_a_step_allocates_nothing(abi, T):
    from sparse_long_context_csa_b200 import harness
    p, x = layer(harness, T)
    o = harness.moe_buffers(p)
    harness.moe_step(p, x, o)                           # the library that PyTorch calls makes its workspace once
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    harness.moe_step(p, x, o)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before


@pytest.mark.parametrize("way", ["stream", "handle", "default"])
def test_a_step_on_a_stream_that_is_not_the_current_one(abi, way):
    """Behind work that keeps the stream busy for a while: nothing of the step may run ahead of it."""
    from sparse_long_context_csa_b200 import harness
    p, x = layer(harness, 300)
    want, o = harness.moe_buffers(p), harness.moe_buffers(p)
    harness.moe_step(p, x, want)
    big = torch.zeros(1 << 28, device="cuda")
    for t in o.values():
        if t is not None:
            t.zero_()
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    where = torch.cuda.default_stream() if way == "default" else side
    with torch.cuda.stream(where):
        for _ in range(20):
            big += 1.0
    with torch.cuda.stream(other):
        harness.moe_step(p, x, o, stream=where if way == "stream" else where.cuda_stream)
    where.synchronize()
    for n in ("stream", "y", "logits", "ids", "weights", "out"):
        assert torch.equal(o[n], want[n]), n


# ------------------------------------------------------------------ no tokens

def test_tensors_of_no_tokens(abi):
    """A batch that is empty: torch's tensors of no rows have no address."""
    from sparse_long_context_csa_b200 import harness
    for eight_bit in (False, True):
        p = harness.moe_params(0, 256, 64, 8, 2, eight_bit=eight_bit)
        o = harness.moe_buffers(p)
        x = dict(attn=torch.empty(0, 256, device="cuda").bfloat16(), stream=torch.empty(0, 256, device="cuda").bfloat16(),
                 gamma=torch.ones(256, device="cuda").bfloat16(), router=torch.zeros(8, 256, device="cuda"), bias=torch.zeros(8, device="cuda"),
                 w13=torch.zeros(8, 128, 256, device="cuda").bfloat16(), w2=torch.zeros(8, 256, 64, device="cuda").bfloat16())
        before = abi.dsv4_launch_count()
        harness.moe_step(p, x, o)
        assert abi.dsv4_launch_count() == before
    torch.cuda.synchronize()


# ------------------------------------------------------------------ a launch that is refused

def test_a_refused_launch_leaves_no_error_behind(tmp_path):
    """The runtime keeps a failed call's error until it is asked for, and the attention's launchers ask
    behind their own launches: an error that stayed would be theirs.  The launch is refused on the host
    (a CTA of more threads than there can be)."""
    import subprocess
    from sparse_long_context_csa_b200 import build
    (tmp_path / "t.cu").write_text("""
#include <stdio.h>
#include "launch.cuh"
namespace dsv4 { void note_launch(int) { printf("launched "); } }
__global__ void nothing(int) {}
int main() {
  const cudaError_t e = dsv4::launch(nothing, 1, 4096, 0, cudaStream_t(nullptr), 1);
  printf("%d %d", e != cudaSuccess, cudaGetLastError() == cudaSuccess);
}
""")
    subprocess.run([build.NVCC, *build._flags(False), str(tmp_path / "t.cu"), "-o", str(tmp_path / "t")], check=True)
    assert subprocess.run([str(tmp_path / "t")], check=True, capture_output=True, text=True).stdout == "1 1"


# ------------------------------------------------------------------ the 8-bit form

@pytest.mark.parametrize("T,hidden", [(2048, 4096), (3000, 333), (900, 5001)])
def test_8_bit_values_are_those_of_the_division(abi, T, hidden):
    """q = e4m3(y / s), bit for bit: float32 rows hand out the y that q is formed from."""
    x = torch.randn(T, hidden, generator=gen(T), device="cuda")
    w = 1 + 0.3 * torch.randn(hidden, generator=gen(T + 1), device="cuda")
    x[::7, 3], w[9], x[5] = -0.0, 0.0, -0.0                        # zeros of both signs
    for pow2 in (0, 1):
        y, q = torch.empty_like(x), torch.empty(T, hidden, dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty(T, -(-hidden // 128), device="cuda")
        abi.dsv4_add_rms_norm(params(abi, T=T, hidden=hidden, scale_pow2=pow2, dtype=abi.F32), x, None, w, None, y, q, s)
        want = (y / s.repeat_interleave(128, 1)[:, :hidden]).clamp(-448, 448).to(torch.float8_e4m3fn)
        wrong = int((q.view(torch.uint8) != want.view(torch.uint8)).sum())
        assert wrong == 0, f"{wrong} of {T * hidden}"


# ------------------------------------------------------------------ weights beside masked logits

def check_weights(abi, logits, bias, fn, topk, n_group=1, topk_group=1, renorm=1, scale=2.5):
    """Ids and weights with a bound per token, from the logits that it chose.  exp's argument is rounded
    by u of itself and by the product with log2(e) once more; arguments beyond 104 (where fp32's exp is
    zero) leave no weight.  A softmax adds the sum's error (argument up to 104 for every term that is
    not zero) and its chain of E / 32 + 16 additions; 40 u are for exp, log1p, the root, the divisions
    and the products, as in the other file; renormalised weights have the error of the sum too."""
    T, E = logits.shape
    p = params(abi, T=T, E=E, topk=topk, n_group=n_group, topk_group=topk_group, score_fn=FN[fn], renorm=renorm, routed_scale=scale,
               logits_dtype=abi.F32 if logits.dtype == torch.float32 else abi.BF16)
    ids, w = torch.empty(T, topk, dtype=torch.int32, device="cuda"), torch.empty(T, topk, device="cuda")
    abi.dsv4_route_experts(p, logits, bias, ids, w)
    l, got = f64(logits), f64(w)
    ref_ids, ref = O.route(l, None if bias is None else f64(bias), fn=fn, topk=topk, n_group=n_group, topk_group=topk_group,
                           renorm=bool(renorm), routed_scale=scale)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids)
    for t in range(T):
        chosen = l[t][ref_ids[t]]
        live = ref[t] > 0
        assert np.all(got[t][~live] == 0), f"token {t}: a weight where there is none"
        if not live.any():
            continue
        arg = chosen[live] - (l[t].max() if fn == "softmax" else 0)
        every = l[t][np.isfinite(l[t])] - l[t].max() if fn == "softmax" else np.zeros(1)
        top = min(np.abs(arg).max(), 104.0) + min(np.abs(every).max(), 104.0)
        rel = 2.0 ** -24 * (40 + 2 * top + E / 32) * (2 if renorm else 1)
        assert np.all(np.abs(got[t] - ref[t])[live] <= rel * ref[t][live]), f"token {t}: {got[t]} instead of {ref[t]}"


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("renorm", [0, 1])
def test_weights_beside_masked_logits(abi, fn, renorm):
    """Rows of -inf, of the lowest value, with fewer experts left than are chosen, and ordinary ones."""
    T, E = 8, 40
    for dt in (torch.float32, torch.bfloat16):
        logits = torch.randn(T, E, generator=gen(8), device="cuda").to(dt)
        logits[0] = -float("inf")
        logits[1, 3:] = -float("inf")
        logits[2] = torch.finfo(dt).min
        logits[3, ::2] = torch.finfo(dt).min
        logits[4, 4:] = torch.finfo(dt).min
        check_weights(abi, logits, None, fn, 6, renorm=renorm)
        check_weights(abi, logits, None, fn, 6, 4, 2, renorm)
        bias = 0.1 * torch.randn(E, generator=gen(9), device="cuda")
        check_weights(abi, logits, bias, fn, 6, renorm=renorm)
        check_weights(abi, logits, bias, fn, 6, 4, 2, renorm)


def test_a_stream_that_is_given(abi):
    """Without ctypes as well: behind work that keeps it busy, while the current stream has none; what is no
    stream's handle is left to the function that says so."""
    T, h = 64, 512
    p = params(abi, T=T, hidden=h)
    x, w = torch.randn(T, h, generator=gen(60), device="cuda").bfloat16(), torch.ones(h, device="cuda").bfloat16()
    want, y = torch.empty_like(x), torch.empty_like(x)
    assert abi._norm(p, x, None, w, None, want, None, None) == 0
    big, side = torch.zeros(1 << 28, device="cuda"), torch.cuda.Stream()
    for way in (side, side.cuda_stream):
        late = torch.zeros_like(x)
        y.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                big += 1.0
            late.copy_(x)
        abi.dsv4_add_rms_norm(p, late, None, w, None, y, stream=way)
        side.synchronize()
        assert torch.equal(y, want)
    assert abi._norm(p, x, None, w, None, y, None, None, side.cuda_stream) == 0
    assert abi._norm(p, x, None, w, None, y, None, None, None) == 0
    assert abi._norm(p, x, None, w, None, y, None, None, 1.5) is None
    assert abi._norm(p, x, None, w, None, y, None, None, 1 << 80) is None
    assert abi._norm(p, x, None, w, None, y, None, None, None, None) is None
    torch.cuda.synchronize()
