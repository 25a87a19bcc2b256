"""nslm_moe_balance and nslm_moe_balance_grad against the formulas in 64 bits.

The tolerance of a probability: z - m is off by half a step of at most 2^5 in
magnitude here, which moves exp by at most 2^5 2^-24 of it; expf itself by 2
steps, the sum of a row by its additions in a lane and over the lanes (at most
37), the quotient by a half step: together below 96 * 2^-24 of the value.  A
mean over tokens adds a half step for each token that one thread sums (at most
T / 8)."""
import numpy as np
import pytest
import torch

import guard

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nslm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lfsr_seeded_moe_b200 import nslm as n
    return n


def _inputs(T, E, k, seed, skew=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    z = torch.randn(T, E, generator=g, device="cuda") + skew * torch.randn(E, generator=g, device="cuda")
    ids = torch.topk(z, k, dim=1).indices.to(torch.int32).contiguous()
    return z, ids


def _want(z, ids, mask, E, k, coef):
    """(counts with n, offsets, mean_p, loss, P) in 64 bits; P: the tokens' probabilities."""
    T = z.shape[0]
    live = np.ones(T, bool) if mask is None else mask.cpu().numpy() != 0
    zz = z.double().cpu().numpy().copy()
    zz[~live] = 0
    m = zz.max(1, keepdims=True) if T else zz.reshape(0, 1)
    dead = np.isneginf(m[:, 0])
    with np.errstate(invalid="ignore"):
        e = np.exp(zz - m)
    e[dead] = 0
    p = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    p[~live] = 0
    picked = ids.cpu().numpy()[live].reshape(-1)
    counts = np.bincount(picked[(picked >= 0) & (picked < E)], minlength=E)
    n = int(live.sum())
    mean = p.sum(0) / max(1, n)
    loss = coef * E * float((counts / (k * max(1, n)) * mean).sum())
    return np.append(counts, n), np.append(0, np.cumsum(counts)), mean, loss, p


def _run(nslm, z, ids, mask, E, k, coef, T=None):
    T = z.shape[0] if T is None else T
    need = nslm.nslm_workspace_bytes(nslm.NSLM_OP_MOE_BALANCE, T, E, 0, 0, k)
    ws = guard.buffer(need, torch.uint8, fill=0xFF) if need else None
    counts = guard.buffer(E + 1, torch.int32, fill=-1)
    offsets = guard.buffer(E + 1, torch.int32, fill=-1)
    mean = guard.buffer(E, torch.float32, fill=float("nan"))
    loss = guard.buffer(1, torch.float32, fill=float("nan"))
    nslm.nslm_moe_balance(z, ids, mask, T, E, k, coef, counts, offsets, mean, loss, ws, need)
    assert nslm.nslm_last_launch_count() == (2 if need else 1)
    return counts, offsets, mean, loss


def _grad(nslm, z, counts, mask, k, coef, dloss):
    T, E = z.shape
    d = guard.buffer((T, E), torch.float32, fill=float("nan"))
    nslm.nslm_moe_balance_grad(z, counts, mask, T, E, k, coef, dloss, d)
    assert nslm.nslm_last_launch_count() == 1
    return d


def _want_grad(p, counts, E, k, coef, dloss):
    n = max(1, int(counts[E]))
    f = counts[:E] / (k * n)
    dot = (p * f).sum(1, keepdims=True)
    d = dloss * coef * E / n * p * (f - dot)
    return d, abs(dloss) * coef * E / n * p * (f + dot)


SHAPES = [(1, 1, 1), (1, 8, 8), (2, 3, 2), (7, 100, 8), (64, 100, 8), (65, 33, 4), (512, 100, 8), (1024, 128, 2),
          (1025, 4, 1), (3000, 100, 8), (5000, 257, 6), (1500, 1024, 8), (20000, 64, 4), (40, 1023, 3), (2500, 130, 8)]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_counts_loss_and_gradient(nslm, T, E, k, masked):
    z, ids = _inputs(T, E, k, T + E)
    mask = None
    if masked:  # padding holds anything
        mask = torch.ones(T + 16, dtype=torch.uint8, device="cuda")[:T].contiguous()
        mask[T // 3::4] = 0
        z[mask == 0] = float("nan")
        ids[mask == 0] = 2**31 - 1
    counts, offsets, mean, loss = _run(nslm, z, ids, mask, E, k, 0.5)
    wc, wo, wm, wl, p = _want(z, ids, mask, E, k, 0.5)
    assert np.array_equal(counts.cpu().numpy(), wc)
    assert np.array_equal(offsets.cpu().numpy(), wo)
    rel = (96 + T // 8) * 2.0 ** -24
    assert np.all(np.abs(mean.cpu().numpy() - wm) <= rel * wm)
    assert abs(float(loss) - wl) <= rel * wl
    dloss = torch.tensor([1.5], device="cuda")
    d = _grad(nslm, z, counts, mask, k, 0.5, dloss).cpu().numpy()
    wd, size = _want_grad(p, wc, E, k, 0.5, 1.5)
    # two probabilities enter a value, one by itself and one in the dot product
    assert np.all(np.abs(d - wd) <= 2 * 96 * 2.0 ** -24 * size + 1e-44)


def test_gradient_against_differences(nslm):
    # central differences of the kernel's own loss: off by h^2/6 of a third
    # derivative below 1 here, and by the loss's half step over h
    T, E, k, coef, h = 3, 6, 2, 1.0, 0.03
    z, ids = _inputs(T, E, k, 77)
    counts, _, _, loss = _run(nslm, z, ids, None, E, k, coef)
    d = _grad(nslm, z, counts, None, k, coef, None)
    for t in range(T):
        for e in range(E):
            at = []
            for sign in (1, -1):
                y = z.clone()
                y[t, e] += sign * h
                at.append(float(_run(nslm, y, ids, None, E, k, coef)[3]))
            tol = h * h / 6 + 2 * 96 * 2.0 ** -24 * float(loss) / h
            assert abs((at[0] - at[1]) / (2 * h) - float(d[t, e])) <= tol, (t, e)


def test_masked_experts_and_empty_rows(nslm):
    # experts that a user took out (-inf), a row with none left, ids that are out of range or listed twice
    T, E, k = 30, 20, 4
    z, ids = _inputs(T, E, k, 5)
    z[:, 7] = -float("inf")
    z[4] = -float("inf")
    ids[0] = torch.tensor([-1, E, 3, 3], dtype=torch.int32)
    counts, offsets, mean, loss = _run(nslm, z, ids, None, E, k, 2.0)
    wc, wo, wm, wl, p = _want(z, ids, None, E, k, 2.0)
    assert np.array_equal(counts.cpu().numpy(), wc) and np.array_equal(offsets.cpu().numpy(), wo)
    rel = (96 + T // 8) * 2.0 ** -24
    assert np.all(np.abs(mean.cpu().numpy() - wm) <= rel * wm) and float(mean[7]) == 0
    assert abs(float(loss) - wl) <= rel * wl
    d = _grad(nslm, z, counts, None, k, 2.0, None).cpu().numpy()
    wd, size = _want_grad(p, wc, E, k, 2.0, 1.0)
    assert np.all(np.abs(d - wd) <= 2 * 96 * 2.0 ** -24 * size + 1e-44)
    assert np.all(d[4] == 0) and np.all(d[:, 7] == 0)


def test_lowest_values_in_masked_places(nslm):
    # a mask of the type's lowest value instead of -inf: probability zero, no overflow into NaN
    z, ids = _inputs(12, 40, 2, 6)
    z[:, 30:] = torch.finfo(torch.float32).min
    ids.clamp_(max=29)
    counts, _, mean, loss = _run(nslm, z, ids, None, 40, 2, 1.0)
    assert bool((mean[30:] == 0).all()) and bool(torch.isfinite(mean).all()) and bool(torch.isfinite(loss).all())
    d = _grad(nslm, z, counts, None, 2, 1.0, None)
    assert bool((d[:, 30:] == 0).all()) and bool(torch.isfinite(d).all())


@pytest.mark.parametrize("T", [0, 5, 3000])
def test_no_token_that_counts(nslm, T):
    z = torch.full((max(T, 1), 16), float("nan"), device="cuda")[:T]
    ids = torch.zeros(max(T, 1), 2, dtype=torch.int32, device="cuda")[:T]
    mask = torch.zeros(max(T, 1), dtype=torch.uint8, device="cuda")
    counts, offsets, mean, loss = _run(nslm, z, ids, mask, 16, 2, 1.0, T)
    assert bool((counts == 0).all()) and bool((offsets == 0).all()) and bool((mean == 0).all()) and float(loss) == 0
    if T:
        assert bool((_grad(nslm, z, counts, mask, 2, 1.0, None) == 0).all())


def test_optional_outputs_and_equal_bits(nslm):
    T, E, k = 4000, 100, 8
    z, ids = _inputs(T, E, k, 8)
    a = _run(nslm, z, ids, None, E, k, 0.1)
    need = nslm.nslm_workspace_bytes(nslm.NSLM_OP_MOE_BALANCE, T, E, 0, 0, k)
    ws = guard.buffer(need, torch.uint8)
    for _ in range(3):
        counts = guard.buffer(E + 1, torch.int32, fill=-1)
        loss = guard.buffer(1, torch.float32, fill=float("nan"))
        nslm.nslm_moe_balance(z, ids, None, T, E, k, 0.1, counts, None, None, loss, ws, need)
        assert torch.equal(counts, a[0]) and torch.equal(loss, a[3])


def test_gradient_in_place_and_counts_of_a_larger_batch(nslm):
    # data-parallel: two halves with the summed counts give the whole batch's gradient, also in place
    T, E, k = 600, 48, 4
    z, ids = _inputs(T, E, k, 12)
    counts = _run(nslm, z, ids, None, E, k, 1.0)[0]
    whole = _grad(nslm, z, counts, None, k, 1.0, None)
    parts = [_run(nslm, z[i:i + 300].contiguous(), ids[i:i + 300].contiguous(), None, E, k, 1.0)[0] for i in (0, 300)]
    both = parts[0] + parts[1]
    assert torch.equal(both, counts)
    for i in (0, 300):
        h = guard.buffer((300, E), torch.float32)
        h.copy_(z[i:i + 300])
        nslm.nslm_moe_balance_grad(h, both, None, 300, E, k, 1.0, None, h)
        assert torch.equal(h, whole[i:i + 300])


def test_even_counts_give_the_coefficient(nslm):
    # equal logits and even counts: loss = coef exactly up to rounding of 1/E
    T, E, k = 32, 8, 2
    z = torch.zeros(T, E, device="cuda")
    ids = (torch.arange(T * k, device="cuda", dtype=torch.int32) % E).reshape(T, k).contiguous()
    counts, _, _, loss = _run(nslm, z, ids, None, E, k, 0.25)
    assert float(loss) == 0.25
    assert bool((_grad(nslm, z, counts, None, k, 0.25, None) == 0).all())


def test_captured_and_replayed(nslm):
    T, E, k = 2000, 64, 4
    z, ids = _inputs(T, E, k, 1)
    need = nslm.nslm_workspace_bytes(nslm.NSLM_OP_MOE_BALANCE, T, E, 0, 0, k)
    ws = guard.buffer(need, torch.uint8)
    counts = guard.buffer(E + 1, torch.int32)
    loss = guard.buffer(1, torch.float32)
    d = guard.buffer((T, E), torch.float32)

    def step():
        nslm.nslm_moe_balance(z, ids, None, T, E, k, 1.0, counts, None, None, loss, ws, need)
        nslm.nslm_moe_balance_grad(z, counts, None, T, E, k, 1.0, loss, d)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (2, 3):
        z2, ids2 = _inputs(T, E, k, seed)
        z.copy_(z2), ids.copy_(ids2)
        step()
        torch.cuda.synchronize()
        a = counts.clone(), loss.clone(), d.clone()
        counts.zero_(), loss.zero_(), d.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a[0], counts) and torch.equal(a[1], loss) and torch.equal(a[2], d)
        wc, _, _, wl, p = _want(z, ids, None, E, k, 1.0)
        assert np.array_equal(counts.cpu().numpy(), wc)
        assert abs(float(loss) - wl) <= (96 + T // 8) * 2.0 ** -24 * wl


def test_offsets_past_32_bits(nslm):
    T, E, k = 2_200_000, 1000, 1  # 8.8 GB of logits
    z = torch.zeros(T, E, device="cuda")
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    mask = torch.zeros(T, dtype=torch.uint8, device="cuda")
    mask[-3:] = 1
    z[-3:, 5] = 3.0
    ids[-3:] = 5
    counts, _, mean, loss = _run(nslm, z, ids, mask, E, k, 1.0)
    p5 = np.exp(3.0) / (np.exp(3.0) + E - 1)
    assert int(counts[5]) == 3 and int(counts[E]) == 3
    assert abs(float(mean[5]) - p5) <= 99 * 2.0 ** -24 * p5
    d = z
    nslm.nslm_moe_balance_grad(z, counts, mask, T, E, k, 1.0, None, d)
    want = E / 3 * p5 * (1 - p5)
    # p5 by itself and in the dot product that is taken from 1
    assert bool(((d[-3:, 5] - want).abs() <= 2 * 96 * 2.0 ** -24 * E / 3 * p5 * (1 + p5)).all())
    assert bool((d[:-3] == 0).all())


def test_graphs_that_share_a_workspace_and_calls_at_once(nslm):
    # one workspace for two captured graphs of unlike sizes, replayed in turn (nothing in it outlives a call);
    # two of its own for calls on two streams at once
    E, k = 100, 8
    z, ids = _inputs(6000, E, k, 41)
    need = nslm.nslm_workspace_bytes(nslm.NSLM_OP_MOE_BALANCE, 6000, E, 0, 0, k)
    ws = [guard.buffer(need, torch.uint8, fill=0xFF) for _ in range(2)]
    out = [(guard.buffer(E + 1, torch.int32, fill=-1), guard.buffer(1, torch.float32)) for _ in range(2)]
    sizes = (6000, 1100)
    want = [_want(z[:T], ids[:T], None, E, k, 1.0) for T in sizes]

    def call(i, w, stream=None):
        nslm.nslm_moe_balance(z, ids, None, sizes[i], E, k, 1.0, out[i][0], None, None, out[i][1], w, need, stream)

    def check():
        for i, T in enumerate(sizes):
            assert np.array_equal(out[i][0].cpu().numpy(), want[i][0])
            assert abs(float(out[i][1]) - want[i][3]) <= (96 + T // 8) * 2.0 ** -24 * want[i][3]
            out[i][0].fill_(-1), out[i][1].zero_()

    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            call(i, ws[0])
    for _ in range(3):
        graphs[0].replay()
        graphs[1].replay()
        check()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            call(i, ws[i], streams[i])
    torch.cuda.synchronize()
    check()


def test_gradient_through_a_graph_while_the_loss_is_used_eagerly(nslm):
    # the gradient captured while an eager call of the same logits is under way: plain buffers, no state between
    T, E, k = 1200, 40, 2
    z, ids = _inputs(T, E, k, 42)
    counts = _run(nslm, z, ids, None, E, k, 1.0)[0]
    want = _grad(nslm, z, counts, None, k, 1.0, None)
    d = guard.buffer((T, E), torch.float32, fill=float("nan"))
    eager = guard.buffer((T, E), torch.float32, fill=float("nan"))
    nslm.nslm_moe_balance_grad(z, counts, None, T, E, k, 1.0, None, eager)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nslm.nslm_moe_balance_grad(z, counts, None, T, E, k, 1.0, None, d)
    g.replay()
    assert torch.equal(d, want) and torch.equal(eager, want)
