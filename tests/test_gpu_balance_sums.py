"""The balance loss's sums over many tokens, with bounds that follow the order
in which the kernel adds.

With h = 2^-24 (half a step of fp32) and M the largest |z - max z| of a row, a
probability is off by
  (3M + 4) h  in its exponential: the difference, log2 e and their product are
              rounded, each moving the result by M h; ex2 is off by two steps,
  as much and 37 h in the row's sum (at most 32 additions in a lane, 5 over the lanes),
  h           in the quotient;
a mean by the additions that follow, each h: a lane's in fp32, of which there are
64 at most before they go on in fp64, 2 over a warp's tokens, 24 over the warps,
and one rounding of a CTA's part and one of the result."""
import math

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


def _in_flight(E):
    """Tokens that the GPU's CTAs take at once: 148 CTAs of 24 warps, 8, 16 or 32 lanes a token."""
    return 148 * 24 * (4 if E <= 128 else 2 if E <= 256 else 1)


def _bound(M, T, E):
    rounds = math.ceil(T / _in_flight(E)) if T > 1024 else 8
    return (2 * (3 * M + 4) + 37 + 1 + min(64, rounds) + 2 + 24 + 2) * 2.0 ** -24


def _run(nslm, z, ids, E, k):
    T = z.shape[0]
    need = nslm.nslm_workspace_bytes(nslm.NSLM_OP_MOE_BALANCE, T, E, 0, 0, k)
    ws = guard.buffer(need, torch.uint8, fill=0xFF) if need else None
    counts = guard.buffer(E + 1, torch.int32, fill=-1)
    mean = guard.buffer(E, torch.float32, fill=float("nan"))
    loss = guard.buffer(1, torch.float32, fill=float("nan"))
    nslm.nslm_moe_balance(z, ids, None, T, E, k, 1.0, counts, None, mean, loss, ws, need)
    return counts.cpu().numpy(), mean.cpu().numpy(), float(loss)


def _mean(z):
    """(mean over the tokens, M) in 64 bits."""
    total, M = 0, 0.0
    for part in z.split(1 << 16):
        y = part.double() - part.double().amax(1, keepdim=True)
        M = max(M, float(-y.min()))
        e = torch.exp(y)
        total = total + (e / e.sum(1, keepdim=True)).sum(0)
    return total.cpu().numpy() / z.shape[0], M


def _check(counts, mean, loss, want, M, T, E, k):
    rel = _bound(M, T, E)
    assert np.all(np.abs(mean - want) <= rel * want), (np.abs(mean / want - 1).max(), rel)
    loss64 = E * float((counts[:E] / (k * T) * want).sum())
    assert abs(loss - loss64) <= rel * loss64


@pytest.mark.parametrize("seed", [0, 2])
def test_thousands_of_equal_tokens_a_lane(nslm, seed):
    # 4,724 tokens a lane whose probabilities are rounded the same way every time
    T, E, k = 1 << 26, 8, 1
    row = torch.from_numpy(np.random.RandomState(seed).randn(1, E).astype(np.float32)).cuda()
    z = row.expand(T, E).contiguous()
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    counts, mean, loss = _run(nslm, z, ids, E, k)
    want, M = _mean(row)
    assert counts[0] == T and counts[E] == T
    _check(counts, mean, loss, want, M, T, E, k)


@pytest.mark.parametrize("T,E,k", [(100_000, 8, 2), (1_000_000, 20, 4), (600_000, 300, 8), (300_000, 1023, 2)])
def test_blocks_of_tokens(nslm, T, E, k):
    # one block of a lane's tokens and several, the last of them short
    g = torch.Generator("cuda").manual_seed(T)
    z = torch.randn(T, E, generator=g, device="cuda")
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    counts, mean, loss = _run(nslm, z, ids, E, k)
    want, M = _mean(z)
    assert np.array_equal(counts[:E], torch.bincount(ids.reshape(-1).long(), minlength=E).cpu().numpy())
    _check(counts, mean, loss, want, M, T, E, k)


@pytest.mark.parametrize("T,E,k", [(64, 100, 8), (513, 1024, 8), (1024, 100, 8), (1025, 64, 2), (14208, 128, 4),
                                   (28417, 100, 4), (65536, 128, 8), (65537, 128, 8), (14209, 200, 4), (10657, 600, 8),
                                   (909313, 64, 1)])
def test_no_token_is_lost_or_counted_twice(nslm, T, E, k):
    # tokens at the ends of rounds and blocks have an expert each to themselves,
    # which then makes most of that expert's mean
    g = torch.Generator("cuda").manual_seed(T)
    F = _in_flight(E)
    at = sorted({t for i in (0, 1, 2, 63, 64) for t in (i * F - 1, i * F) if 0 <= t < T} | {0, T // 2, T - 1})
    z = torch.randn(T, E, generator=g, device="cuda")
    z[:, :len(at)] -= 8
    for e, t in enumerate(at):
        z[t, e] = 12
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    counts, mean, loss = _run(nslm, z, ids, E, k)
    want, M = _mean(z)
    rel = _bound(M, T, E)
    assert np.all(want[:len(at)] * T * rel < 0.1)  # a token more or less would be seen
    _check(counts, mean, loss, want, M, T, E, k)


@pytest.mark.parametrize("E,k", [(8, 8), (100, 8), (1023, 2)])
def test_gradient_with_counts_of_many_ranks(nslm, E, k):
    # counts summed over ranks: each below 2^31, their total far above, and nearly
    # even, so that nothing is left of their differences unless their mean is taken
    # off first.  f_e less the mean is rounded once; with it a value has the errors
    # of two probabilities (each (2 (3M + 4) + 38) h) and of the dot product's sum
    # (37 h), its centring (h) and five products.
    T = 9
    g = torch.Generator("cuda").manual_seed(E)
    z = torch.randn(T, E, generator=g, device="cuda")
    c = 2**30 + torch.randint(-2000, 2000, (E,), generator=g, device="cuda")
    assert int(c.sum()) > 2**31
    n = min(int(c.sum()) // k, 2**31 - 1)
    counts = torch.cat([c, c.new_tensor([n])]).to(torch.int32)
    d = guard.buffer((T, E), torch.float32, fill=float("nan"))
    nslm.nslm_moe_balance_grad(z, counts, None, T, E, k, 0.5, None, d)
    y = z.double() - z.double().amax(1, keepdim=True)
    p = torch.exp(y) / torch.exp(y).sum(1, keepdim=True)
    f = (c.double() - c.double().mean()) / (k * n)
    scale = 0.5 * E / n
    want = scale * p * (f - (p * f).sum(1, keepdim=True))
    size = scale * p * (f.abs() + (p * f.abs()).sum(1, keepdim=True))
    rel = (2 * (2 * (3 * float(-y.min()) + 4) + 38) + 37 + 1 + 5) * 2.0 ** -24
    assert bool(((d.double() - want).abs() <= rel * size + 1e-44).all()), float(((d.double() - want).abs() / size).max())
