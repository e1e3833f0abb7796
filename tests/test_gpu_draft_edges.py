"""The drafter's calls at the edges of what their documentation allows: lists without entries,
log-sum-exps that do not belong to their list, temperatures near the smallest number, several host
threads, outputs left out. Tolerances stand beside each test."""
from __future__ import annotations

import ctypes
import math
import threading

import numpy as np
import pytest
import torch

import draft_token_verification_spec_b200 as sv
from tests import _draft_ref as ref
from tests.test_gpu_distill import check, teacher
from tests.test_gpu_sample import check_sample, check_top, make, uniforms

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------------- distillation
@pytest.mark.parametrize("rows", [6, 200])
@pytest.mark.parametrize("V,dtype", [(3000, F32), (40000, BF16), (150000, F32)])
def test_a_list_without_entries_costs_nothing(V, dtype, rows):
    """Exactly nothing, in one call as in two, whatever the row's log-sum-exp is."""
    if V == 150000:
        rows = min(rows, 20)
    x = make(rows, V, dtype)
    ids, val, lse = teacher(x, 12, short=False)
    ids[:rows // 2] = -1
    val[rows // 2:] = -math.inf
    for l in (None, lse):
        loss, _ = sv.spec_distill_loss(x, ids, val, l)
        both_loss, grad = sv.spec_distill_loss_grad(x, ids, val, l)
        assert (loss == 0.0).all() and (both_loss == 0.0).all() and (grad == 0.0).all()
    x[1, 5] = math.nan               # still a row in error
    loss, grad = sv.spec_distill_loss_grad(x, ids, val, lse)
    assert torch.isnan(loss[1]) and torch.isnan(grad[1].float()).all() and (loss[2:] == 0.0).all()


def loss_and_gradient(z, ids, val, lse, T):
    """The loss over the whole vocabulary in double, its gradient by automatic differentiation, and
    what the gradient's roundings are relative to (lists without padding)."""
    z = z.double().cpu().requires_grad_(True)
    at, a = ids.cpu().long(), val.double().cpu() / T
    t = (a - lse.double().cpu()[:, None]).exp()
    on = torch.zeros_like(z, dtype=torch.bool).scatter(1, at, True)
    rho = 1.0 - t.sum(1)
    rho = torch.where(rho > (lse.double().cpu().abs() + 1.0) * 2.0 ** -23, rho, 0.0)
    logs = torch.log_softmax(z / T, 1)
    log_sigma = torch.logsumexp(torch.where(on, -math.inf, logs), 1)
    loss = (torch.xlogy(t, t) - t * logs.gather(1, at)).sum(1) + torch.xlogy(rho, rho) - rho * log_sigma
    loss.sum().backward()
    s = logs.detach().exp()
    M = (t.sum(1) + rho)[:, None]
    share = s / log_sigma.detach().exp()[:, None]
    scale = torch.where(on, M * s + torch.zeros_like(s).scatter(1, at, t), M * s + rho[:, None] * share) / T
    return loss.detach(), z.grad, scale


@pytest.mark.parametrize("rows", [4, 180])
@pytest.mark.parametrize("V,dtype,T,off", [(500, F32, 1.3, -0.3), (20000, BF16, 1.0, -1.5),
                                           (30000, F32, 0.7, 0.4), (270000, BF16, 1.0, -0.2)])
def test_a_log_sum_exp_that_is_not_the_list_s_own(V, dtype, T, off, rows):
    """Masses of exp(-off) in all, with and without a rest: the loss counts them as they are, the
    gradient as if they were 1, as the header states. Tolerances as in test_gpu_distill.py: the loss
    1e-5 (1 + M), the gradient 1e-5 of M s + t."""
    if V == 270000:
        rows = min(rows, 4)
    x = make(rows, V, dtype)
    ids, val, _ = teacher(x, 20, short=False, T=T)
    lse = torch.logsumexp(val.double() / T, 1).float() + off
    rl, rg, scale = loss_and_gradient(x, ids, val, lse, T)
    M = (val.double().cpu() / T - lse.double().cpu()[:, None]).exp().sum(1).clamp(min=1.0)
    rg = rg - (M - 1.0)[:, None] * torch.softmax(x.double().cpu() / T, 1) / T
    loss, stats = sv.spec_distill_loss(x, ids, val, lse, T)
    both_loss, both_grad = sv.spec_distill_loss_grad(x, ids, val, lse, T)
    grad = sv.spec_distill_grad(x, ids, val, lse, T, stats)
    step = torch.finfo(dtype).eps / 2
    for got in (loss, both_loss):
        lim = 1e-5 * (1 + M) + 2.0 ** -23 * rl.abs()
        assert ((got.double().cpu() - rl).abs() <= lim).all()
    for got in (grad, both_grad):
        lim = step * rg.abs() + (1 + step) * 1e-5 * scale + 2e-38
        assert ((got.double().cpu() - rg).abs() <= lim).all()


# ------------------------------------------------------------------------- the log-sum-exp of top logits
def few_allowed(rows, V, dtype, keep, kind, seed=0):
    """Rows of which `keep` tokens are allowed: anywhere, or side by side; the others -inf, the type's
    lowest value, or far down."""
    g = torch.Generator().manual_seed(seed * 7 + V)
    x = torch.randn((rows, V), generator=g) * 2.0
    if kind.startswith("beside"):
        first = torch.randint(0, V - keep + 1, (rows, 1), generator=g)
        col = torch.arange(V)[None]
        on = (col >= first) & (col < first + keep)
    else:
        on = torch.zeros((rows, V), dtype=torch.bool)
        for r in range(rows):
            on[r, torch.randperm(V, generator=g)[:keep]] = True
    if kind.endswith("far"):
        return torch.where(on, x, x - 70.0).to(dtype).cuda(), on.cuda()
    out = -math.inf if kind.endswith("masked") else torch.finfo(dtype).min
    x = torch.where(on, x, out)
    if kind.startswith("log"):
        x = torch.where(on, torch.log_softmax(torch.where(on, x, -math.inf), 1), out)
    return x.to(dtype).cuda(), on.cuda()


@pytest.mark.parametrize("rows", [3, 60, 470])
@pytest.mark.parametrize("V,dtype,k,keep,kind,T", [
    (300, F32, 64, 64, "log masked", 1.0), (300, F32, 256, 200, "log lowest", 1.0),
    (33000, BF16, 64, 40, "masked", 0.7), (33000, BF16, 64, 64, "lowest", 1.0),
    (20000, F32, 256, 256, "log masked", 1.0), (70000, BF16, 256, 200, "beside masked", 1.0),
    (40000, F32, 256, 250, "beside far", 1.0), (70000, BF16, 256, 250, "beside far", 1.3),
    (200, F32, 200, 200, "log masked", 1.0), (40000, BF16, 50, 400, "far", 1.0)])
def test_top_logits_log_sum_exp_is_exact_where_the_list_holds_the_mass(rows, V, dtype, k, keep, kind, T):
    """Off by its rounding to float32 (half a step, 2^-24 of itself) and by its sum's float32 weights:
    9e-7 and 8.3e-8 log2 V of the sum (2.6e-6), of which at most 1/128 counts (2.1e-8) where the list
    leaves less than 9e-7 of the mass."""
    x, _ = few_allowed(rows, V, dtype, keep, kind)
    ids, val, lse = sv.spec_top_logits(x, k, T)
    T = float(np.float32(T))
    want = torch.logsumexp(x.double() / T, 1)
    outside = 1.0 - (val.double() / T - want[:, None]).exp().sum(1)
    lim = 2.0 ** -24 * want.abs() + torch.where(outside < 9e-7, 2.1e-8, 2.6e-6)
    assert ((lse.double() - want).abs() <= lim).all(), ((lse.double() - want).abs() / lim).max()
    top = torch.sort(x.float(), dim=1, descending=True, stable=True)
    torch.testing.assert_close(val, top.values[:, :k], rtol=0, atol=0)
    real = top.values[:, :k] > -math.inf
    assert torch.equal(ids, torch.where(real, top.indices[:, :k], -1).to(torch.int32))


@pytest.mark.parametrize("rows,V,keep,k,kind", [(4000, 300, 40, 64, "log masked"), (3000, 200, 200, 200, "log masked"),
                                                (12, 30000, 100, 128, "log masked")])
def test_top_logits_that_hold_all_the_mass_leave_no_rest(rows, V, keep, k, kind):
    """A teacher and a student that allow the same tokens, all of them listed: the student has no
    mass outside the list, and with the list's own log-sum-exp the teacher has none there either."""
    t, on = few_allowed(rows, V, F32, keep, kind)
    ids, val, lse = sv.spec_top_logits(t, k, 1.0)
    g = torch.Generator().manual_seed(1)
    x = torch.where(on, torch.randn((rows, V), generator=g).cuda(), -math.inf)
    loss, stats = sv.spec_distill_loss(x, ids, val, lse, 1.0)
    grad = sv.spec_distill_grad(x, ids, val, lse, 1.0, stats)
    both_loss, both_grad = sv.spec_distill_loss_grad(x, ids, val, lse, 1.0)
    for got in (loss, both_loss, grad, both_grad):
        assert torch.isfinite(got).all()
    check(x[:200], ids[:200], val[:200], lse[:200])


@pytest.mark.parametrize("rows", [4, 470])
def test_top_logits_are_deterministic(rows):
    """Bit for bit, whatever order the lists were filled in."""
    x = make(rows, 40000, BF16, "zipf")
    first = None
    for _ in range(6):
        got = sv.spec_top_logits(x, 64, 1.0)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


# ------------------------------------------------------------------------- temperatures near nothing
@pytest.mark.parametrize("T", [1e-37, 3e-35, 1e-33, 1e-31])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_logits_and_temperatures_near_the_smallest_number(T, dtype):
    """Weights depend on the logits' differences over the temperature alone, however small both are.
    Tolerances as in the calls' own tests. (The logits of the smallest are normal numbers but for
    those within 0.1 of nothing, held to 1e-7 of T.)"""
    x = make(5, 900, F32).mul(T).to(dtype)
    u = uniforms(5)
    for st in (dict(), dict(k=30), dict(p=0.9), dict(q=0.1), dict(k=200, p=0.8, q=0.001)):
        check_sample(x, u, T, **st)
    row_T = torch.full((5,), T, device="cuda")
    check_sample(x, u, row_T, 0, 0.9)
    check_top(x, 20, T)
    ids, val, lse = teacher(x, 20, T=T, spread=2.0 * T)
    check(x, ids, val, lse, T, torch.full((5,), T, device="cuda"))     # (gradients of (s - t) T / T)
    check(x, ids, val, None, T, torch.full((5,), T, device="cuda"))
    y = make(5, 40000, F32).mul(T).to(dtype)       # rows of several tiles, nuclei longer than a pool
    check_sample(y, u, T, 0, 0.99)
    check_sample(y, u, T)
    check_top(y, 100, T)


@pytest.mark.parametrize("rows,V,dtype", [(3, 5000, F32), (200, 5000, BF16), (60, 40000, BF16), (2, 150000, F32)])
def test_teacher_masses_of_nothing_ask_for_nothing(rows, V, dtype):
    """A log-sum-exp so far above the list that its masses are 0 in double: all mass lies outside, and
    a listed token that the student cannot give costs nothing. The loss is -log sigma, within the 1e-5
    of test_gpu_distill.py."""
    x = make(rows, V, dtype)
    ids, val, lse = teacher(x, 8, short=False)
    x[0, ids[0].long()] = -math.inf
    lse = torch.where(torch.arange(rows, device="cuda") % 3 == 2, lse, 2000.0)
    loss, _, _ = check(x, ids, val, lse)
    off = x.double().scatter(1, ids.long(), -math.inf)
    want = torch.logsumexp(x.double(), 1) - torch.logsumexp(off, 1)
    far = lse == 2000.0
    assert ((loss.double() - want)[far].abs() < 1e-5).all()


@pytest.mark.parametrize("rows,V,dtype", [(5, 3000, F32), (200, 3000, BF16), (60, 40000, BF16), (2, 150000, F32)])
@pytest.mark.parametrize("T", [1e-39, 1.0, 3e38])
def test_no_gradient_is_asked_of_some_rows(rows, V, dtype, T):
    """grad_loss 0 gives gradient 0 at every temperature, whatever the row holds."""
    x = make(rows, V, dtype)
    ids, val, lse = teacher(x, 8)
    g = (torch.arange(rows, device="cuda") % 2).float()
    x[0, 3] = math.nan
    x[2 % rows, 4] = math.inf
    _, stats = sv.spec_distill_loss(x, ids, val, lse, T)
    grads = [sv.spec_distill_grad(x, ids, val, lse, T, stats, g),
             sv.spec_distill_loss_grad(x, ids, val, lse, T, g)[1]]
    for grad in grads:
        assert (grad[::2] == 0.0).all()


# ------------------------------------------------------------------------- several host threads
def hammer(calls, times):
    """Each call (a function of the C ABI and its arguments; the interpreter's lock is released inside)
    over and over on a thread and a stream of its own. Returns the statuses that were not 0."""
    bad = []

    def run(fn, make_args):
        stream = torch.cuda.Stream()
        args = make_args() + [ctypes.c_void_p(stream.cuda_stream)]
        torch.cuda.synchronize()
        for i in range(times):
            st = fn(*args)
            if st:
                bad.append(st)
            if i % 200 == 199:
                stream.synchronize()

    threads = [threading.Thread(target=run, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return bad


def test_calls_of_different_pools_from_several_threads():
    """Calls whose finishing takes different amounts of shared memory, at once: what one asks for must
    not be taken away by another before it launches."""
    R, V = 1, 500000
    x, u = make(R, V, BF16), uniforms(R)
    lib, p = sv.lib(), lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    kept = []

    def sample(k, top_p):
        def args():
            n = sv.spec_sample_workspace_size(R, V)
            ws = torch.empty(n, dtype=torch.uint8, device="cuda")
            tok = torch.empty(R, dtype=torch.int32, device="cuda")
            kept.append((k, top_p, tok, ws))
            return [p(x), 1, R, V, V, p(u), 1.0, k, top_p, 0.0, None, None, None, None, p(tok), None,
                    p(ws), n]
        return args

    calls = [(lib.spec_sample, sample(*kw)) for kw in ((256, 1.0), (0, 0.9), (256, 0.8), (0, 0.7))]
    assert hammer(calls, 20000) == []
    for k, top_p, tok, _ in kept:
        assert tok.tolist() == ref.sample_rows(x, u, 1.0, k, top_p, 0.0)[0].tolist()


def test_linear_state_factors_of_different_lengths_from_several_threads():
    """The same of the state's factors: rounds of 1 and of 32 steps at once."""
    B, H, dk, dv = 1, 1, 256, 8
    lib, p = sv.lib(), lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    g = torch.Generator().manual_seed(2)
    kept = []

    def factors(S):
        def args():
            alpha, beta = (torch.rand((B, H, S), generator=g).cuda() * 0.1 + 0.9 for _ in range(2))
            keys = torch.nn.functional.normalize(torch.randn((B, H, S, dk), generator=g), dim=3).cuda()
            values = torch.randn((B, H, S, dv), generator=g).cuda()
            out = [torch.empty_like(keys), torch.empty_like(values), torch.empty_like(alpha)]
            kept.append((alpha, beta, keys, values, out))
            return [p(alpha), p(beta), p(keys), p(values), B, H, S, dk, dv] + [p(o) for o in out]
        return args

    fn = lib.spec_linear_state_factors
    assert hammer([(fn, factors(S)) for S in (32, 1, 32, 17)], 20000) == []
    for *inputs, out in kept:
        for a, b in zip(out, sv.spec_linear_state_factors(*inputs)):
            assert torch.equal(a, b)


# ------------------------------------------------------------------------- the binding
def test_counts_past_a_c_int():
    """top_k past the range keeps all, as any top_k >= V; k past the limit is refused before its
    outputs are made."""
    x, u = make(3, 500, F32), uniforms(3)
    want = sv.spec_sample(x, u)
    for top_k in (2 ** 31, 2 ** 32 + 1, 2 ** 63, -2 ** 40):
        got = sv.spec_sample(x, u, top_k=top_k)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    wide = torch.zeros((2048, 300), device="cuda")
    before = torch.cuda.max_memory_allocated()
    for k, status in ((257, -2), (2 ** 20, -1), (2 ** 31 - 1, -1), (2 ** 32 + 5, -1), (0, -1), (-3, -1), (-2 ** 40, -1)):
        with pytest.raises(sv.SpecError) as e:
            sv.spec_top_logits(wide, k)
        assert e.value.status == status
    assert torch.cuda.max_memory_allocated() - before < 64 << 20


@pytest.mark.parametrize("call", ["grad", "loss_grad"])
def test_logits_that_require_a_gradient(call):
    """Results carry no graph; the gradient goes on by logits.backward(grad), the logits' own memory
    taken for it too, and a graph that needs the logits it replaced says so."""
    h = torch.randn((4, 32), device="cuda", requires_grad=True)
    w = torch.randn((32, 1000), device="cuda")
    ids, val, lse = teacher(make(4, 1000, F32), 10)

    def gradient(z, out=None):
        if call == "loss_grad":
            loss, grad = sv.spec_distill_loss_grad(z, ids, val, lse, 1.0, grad=out)
            assert not loss.requires_grad
            return grad
        loss, stats = sv.spec_distill_loss(z, ids, val, lse, 1.0)
        assert not loss.requires_grad and not stats.requires_grad
        return sv.spec_distill_grad(z, ids, val, lse, 1.0, stats, grad=out)

    z = h @ w
    grad = gradient(z)
    assert not grad.requires_grad
    z.backward(grad)
    want = grad @ w.T
    torch.testing.assert_close(h.grad, want)
    h.grad = None
    z = h @ w                      # (a product does not keep its result)
    grad = gradient(z, z.detach())
    z.backward(grad)
    torch.testing.assert_close(h.grad, want)
    y = (h @ w).exp()              # (an exponential does)
    gradient(y.detach().log(), y.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    with torch.inference_mode():
        z = make(4, 1000, F32)
        assert torch.isfinite(gradient(z, z)).all()


# ------------------------------------------------------------------------- what the header says of outputs
@pytest.mark.parametrize("rows,V,dtype,kind,T", [
    (64, 128256, BF16, "flat", 1.0), (40, 32003, F32, "equal", 1.0), (600, 16384, BF16, "flat", 2.0),
    (64, 50000, BF16, "normal", 4.0), (12, 151936, BF16, "zipf", 0.7)])
def test_probabilities_of_untruncated_draws(rows, V, dtype, kind, T):
    """A draw without truncation divides a double weight by the row's sum of float32 weights. Each is
    within 2^-22 (ex2) and 2^-23 y ln 2 of itself, y its distance from the largest in bits, whose mean
    over the mass is at most log2(V / S); a warp adds up to 2,048 of them (8 vectors of 8 for each of
    32 lanes) in a tree of 3 + 3 + 5 levels, 2^-24 each, and what follows is in double. Rounded once."""
    x, u = make(rows, V, dtype, kind), uniforms(rows)
    tok, prob = sv.spec_sample(x, u, T)
    rt, rp, _ = ref.sample_rows(x, u, T, 0, 1.0, 0.0)
    z = ref.as_f64(x) / float(np.float32(T))
    S = np.exp(z - z.max(1, keepdims=True)).sum(1)
    lim = 2.0 ** -22 + 11 * 2.0 ** -24 + 2.0 ** -23 * math.log(2.0) * np.log2(V / S) + 2.0 ** -24 + 1e-8
    np.testing.assert_array_equal(tok.cpu().numpy(), rt)
    assert (np.abs(prob.cpu().numpy() / rp - 1.0) <= lim).all()


@pytest.mark.parametrize("rows", [3, 60, 470])
def test_outputs_left_out(rows):
    """The C ABI's optional outputs as NULL: the others are what they are with them."""
    V, k = 20000, 30
    x, u = make(rows, V, BF16, "zipf"), uniforms(rows)
    lib, p = sv.lib(), lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    ws = torch.empty(sv.spec_sample_workspace_size(rows, V), dtype=torch.uint8, device="cuda")
    for top_k, top_p in ((0, 1.0), (k, 1.0), (0, 0.9)):
        tok = torch.empty(rows, dtype=torch.int32, device="cuda")
        assert lib.spec_sample(p(x), 1, rows, V, V, p(u), 1.0, top_k, top_p, 0.0, None, None, None, None,
                               p(tok), None, p(ws), ws.numel(), stream) == 0
        assert torch.equal(tok, sv.spec_sample(x, u, 1.0, top_k, top_p)[0])
    ids = torch.empty((rows, k), dtype=torch.int32, device="cuda")
    val = torch.empty((rows, k), device="cuda")
    ws = torch.empty(sv.spec_top_logits_workspace_size(rows, V, k), dtype=torch.uint8, device="cuda")
    assert lib.spec_top_logits(p(x), 1, rows, V, V, k, 1.0, p(ids), p(val), None, p(ws), ws.numel(),
                               stream) == 0
    want = sv.spec_top_logits(x, k, 1.0)
    assert torch.equal(ids, want[0]) and torch.equal(val, want[1])


def test_many_rows_of_the_deep_kernel():
    """Rows that their lists do not settle, by the thousands and few among thousands (each block takes
    one by itself there, a cluster one here), on both sides of the 2,048 that are listed at a time."""
    rows, V = 4500, 2000
    x, u = make(rows, V, BF16, "normal"), uniforms(rows)
    few = [5, 2047, 2048, 2050, 4097, 4499]
    for deep in (few, list(range(2048)) + few, list(range(2100, 4500)), list(range(rows))):
        k = torch.full((rows,), 20, dtype=torch.int32)
        k[deep] = 1500
        check_sample(x, u, 0.9, k.cuda(), 0.95, 0.0)
        y = x.clone()
        y[deep] = torch.round(y[deep] * 0.2)          # a few hundred equal entries at every threshold
        check_top(y, 100)
        check_sample(y, u, 1.0, 100)


# ------------------------------------------------------------------------- sizes
def test_rows_further_apart_than_32_bits():
    """Three rows whose starts lie 2.4 GB apart: the same as next to one another, gradients too."""
    V, k, apart = 70001, 40, 1200000007
    x = make(3, V, BF16, "zipf")
    far = torch.empty(2 * apart + V + 5, dtype=BF16, device="cuda")[5:].as_strided((3, V), (apart, 1))
    far.copy_(x)
    u = uniforms(3)
    for st in (dict(), dict(k=50), dict(p=0.9), dict(T=0.0), dict(k=9000)):
        check_sample(far, u, **st)
    check_top(far, k)
    ids, val, lse = teacher(x, k)
    loss, stats = sv.spec_distill_loss(far, ids, val, lse)
    assert torch.equal(loss, sv.spec_distill_loss(x, ids, val, lse)[0])
    want = sv.spec_distill_grad(x, ids, val, lse, 1.0, stats)
    both = sv.spec_distill_loss_grad(x, ids, val, lse)[1]
    assert torch.equal(sv.spec_distill_loss_grad(far, ids, val, lse, grad=far)[1], both)
    far.copy_(x)
    assert torch.equal(sv.spec_distill_grad(far, ids, val, lse, 1.0, stats, grad=far), want)


def test_more_entries_than_32_bits_count():
    """36,000 rows of 128,256 entries, and lists and gradients of as many: the last rows come out as
    they do by themselves."""
    R, V, k, few = 36000, 128256, 64, 40
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.empty((R, V), dtype=BF16, device="cuda")
    x[:-few].normal_(0.0, 3.0, generator=g)
    x[-few:] = make(few, V, BF16, "zipf")
    u = torch.rand(R, generator=g, device="cuda")
    for top_k, top_p in ((50, 1.0), (0, 0.9), (0, 1.0)):
        tok, prob = sv.spec_sample(x, u, 0.8, top_k, top_p)
        rt, rp, _ = ref.sample_rows(x[-few:], u[-few:], 0.8, top_k, top_p, 0.0)
        np.testing.assert_array_equal(tok[-few:].cpu().numpy(), rt)
        np.testing.assert_allclose(prob[-few:].cpu().numpy(), rp, rtol=4e-6)
    ids, val, lse = sv.spec_top_logits(x, k)
    ri, rv, rl = ref.top_rows(x[-few:], k, 1.0)
    np.testing.assert_array_equal(ids[-few:].cpu().numpy(), ri)
    np.testing.assert_array_equal(val[-few:].cpu().numpy(), rv)
    np.testing.assert_allclose(lse[-few:].cpu().numpy(), rl, rtol=2.0 ** -23, atol=2.6e-6)
    i2, v2, l2 = teacher(x[-few:], k)
    ids[-few:], val[-few:], lse[-few:] = i2, v2, l2
    loss, stats = sv.spec_distill_loss(x, ids, val, lse)
    grads = [sv.spec_distill_grad(x, ids, val, lse, 1.0, stats)[-few:].clone()]
    both_loss, grad = sv.spec_distill_loss_grad(x, ids, val, lse, grad=x)
    grads.append(grad[-few:])
    rl, rg, scale = ref.distill_rows(make(few, V, BF16, "zipf"), i2, v2, l2, 1.0)
    for got in (loss, both_loss):
        np.testing.assert_allclose(got[-few:].cpu().numpy(), rl, rtol=2.0 ** -23, atol=1e-5)
    for got in grads:
        assert (np.abs(ref.as_f64(got) - rg) <= 2.0 ** -8 * np.abs(rg) + 1.01e-5 * scale + 2e-38).all()


@pytest.mark.parametrize("rows", [3, 200])
@pytest.mark.parametrize("V,dtype", [(5, F32), (100, BF16), (9003, BF16), (150001, F32)])
def test_lists_longer_than_the_row_and_gradients_over_rows_apart(V, dtype, rows):
    """Lists padded past the vocabulary, the entries in any places; the gradient over logits that are
    cut out of wider rows, whose other entries stay."""
    if V == 150001:
        rows = 3
    k = min(V, 30)
    x = make(rows, V, dtype, "normal")
    ids, val, lse = teacher(x, k, short=False)
    wide_ids = torch.full((rows, 256), -1, dtype=torch.int32, device="cuda")
    wide_val = torch.full((rows, 256), math.nan, device="cuda")     # (beside a negative id: not looked at)
    at = torch.randperm(256, generator=torch.Generator().manual_seed(V))[:k].cuda()
    wide_ids[:, at], wide_val[:, at] = ids, val
    rl, rg, scale = ref.distill_rows(x, ids, val, lse, 1.0)
    loss, stats = sv.spec_distill_loss(x, wide_ids, wide_val, lse)
    step = torch.finfo(dtype).eps / 2
    for call in ("grad", "both"):
        full = torch.full((rows, V + 11), 7.0, dtype=dtype, device="cuda")
        z = full[:, 3:V + 3]
        z.copy_(x)
        if call == "grad":
            grad, got = sv.spec_distill_grad(z, wide_ids, wide_val, lse, 1.0, stats, grad=z), loss
        else:
            got, grad = sv.spec_distill_loss_grad(z, wide_ids, wide_val, lse, grad=z)
        assert grad.data_ptr() == z.data_ptr()
        assert (full[:, :3] == 7.0).all() and (full[:, V + 3:] == 7.0).all()
        np.testing.assert_allclose(got.cpu().numpy(), rl, rtol=2.0 ** -23, atol=1e-5)
        assert (np.abs(ref.as_f64(grad) - rg) <= step * np.abs(rg) + (1 + step) * 1e-5 * scale + 2e-38).all()


def test_streams():
    """A stream as an object or by its handle, the default one's 0 too; one of another device is
    refused, not left aside."""
    x, u = make(5, 30000, BF16, "zipf"), uniforms(5)
    want = sv.spec_sample(x, u, 0.8, 40)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0, torch.cuda.current_stream(), torch.cuda.default_stream()):
        got = sv.spec_sample(x, u, 0.8, 40, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(ValueError, match="stream must be one of"):
        sv._there(lambda: None, side, torch.device("cuda", side.device.index + 1), ())
