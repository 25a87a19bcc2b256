"""nslm_sample where the threshold lies among logits that differ by next to
nothing, or by all magnitudes at once: the search takes few rounds whatever the
values are, so such a row costs about what any other does.

Tokens are compared as in the other tests of sampling: both sides decide by
sums that are off by less than 2^-28 of the total."""
import numpy as np
import pytest
import torch

import guard

pytestmark = pytest.mark.gpu

V = 262144
# A search that took a round for every distinct value would need seconds here;
# six rounds over one row of this length are some hundred microseconds.
LIMIT_MS = 5.0


@pytest.fixture(scope="module")
def nslm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lfsr_seeded_moe_b200 import nslm as n
    return n


def _want(l, u, t, top_k, top_p):
    """(token, prob) of one row in 64 bits."""
    w = np.exp((l - l.max()) / t)
    order = np.argsort(-l, kind="stable")
    n = top_k or len(l)
    if top_p < 1:
        c = np.cumsum(w[order[:n]])
        n = int(np.count_nonzero(c < top_p * c[-1])) + 1
    keep = np.sort(order[:n])
    c = np.cumsum(w[keep])
    i = int(np.count_nonzero(c <= u * c[-1]))
    return int(keep[i]), float(w[keep[i]] / c[-1])


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _distinct(scale):
    return lambda: torch.randperm(V, generator=_gen(1), device="cuda").float() * 2.0 ** -70 * (scale * 2.0 ** 70)


def _both_signs():
    return (torch.randperm(V, generator=_gen(2), device="cuda").float() - V // 2) * 2.0 ** -70 * 2.0 ** -66


def _magnitudes():
    e = torch.randint(0, 150, (V,), generator=_gen(3), device="cuda").double()
    return -((1 + torch.rand(V, generator=_gen(4), device="cuda").double()) * 2.0 ** -e).float()


ROWS = {
    "subnormal": _distinct(2.0 ** -149),     # every fp32 value from 0 to 2^-131
    "tiny": _distinct(2.0 ** -136),          # 2^18 values below 3.1e-36
    "both signs": _both_signs,               # 2^18 values around 0, within 1.6e-36
    "magnitudes": _magnitudes,               # from 2 down to the smallest
}


@pytest.mark.parametrize("t", [1.0, 1e-36])
@pytest.mark.parametrize("row", sorted(ROWS))
def test_thresholds_among_values_that_hardly_differ(nslm, row, t):
    l = ROWS[row]().reshape(1, V)
    host = l[0].double().cpu().numpy()
    u = torch.rand(1, generator=_gen(5), device="cuda")
    temp = torch.full((1,), t, device="cuda")
    token = guard.buffer(1, torch.int32, fill=-7)
    prob = guard.buffer(1, torch.float32, fill=float("nan"))
    for top_k, top_p in ((0, 0.9), (100000, 1.0), (3000, 1.0), (200000, 0.7)):
        k = torch.full((1,), top_k, dtype=torch.int32, device="cuda")
        p = torch.full((1,), top_p, device="cuda")
        params = nslm.sample_params(temp, k, p, None)
        times = []
        for _ in range(3):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            nslm.nslm_sample(l, nslm.NSLM_TYPE_F32, 1, V, V, params, u, token, prob)
            end.record()
            end.synchronize()
            times.append(start.elapsed_time(end))
        want = _want(host, float(u), float(temp), top_k, float(p))
        assert int(token) == want[0], (top_k, top_p)
        assert abs(float(prob) - want[1]) <= (2.0 ** -24 + 2.0 ** -29) * want[1]
        assert min(times) < LIMIT_MS, (top_k, top_p, times)


def test_a_batch_of_such_rows(nslm):
    # more rows than run at once, which pass through rings instead of staying in shared memory
    B, W = 70, 131072
    l = torch.stack([(torch.randperm(W, generator=_gen(i), device="cuda").float() * 2.0 ** -70) * 2.0 ** -66
                     for i in range(B)])
    host = l.double().cpu().numpy()
    u = torch.rand(B, generator=_gen(6), device="cuda")
    p = torch.full((B,), 0.8, device="cuda")
    token = guard.buffer(B, torch.int32, fill=-7)
    nslm.nslm_sample(l, nslm.NSLM_TYPE_F32, B, W, W, nslm.sample_params(None, None, p, None), u, token)
    want = [_want(host[i], float(u[i]), 1.0, 0, float(p[i]))[0] for i in range(B)]
    assert token.cpu().tolist() == want
