"""nslm_sample against its definition in 64 bits.

Tokens have to be equal.  Both sides decide by sums that are off by less than
2^-28 of the total (the kernel rounds each weight to 2^-45, the oracle sums in
fp64), so a random number would have to fall within that of a border between
two tokens to part them.  prob is one fp32 rounding of a quotient whose parts
are off by less than 2^-30."""
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


def _one(l, u, t=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, prob) of one row in 64 bits."""
    l = l.astype(np.float64).copy()
    l[np.isnan(l)] = -np.inf
    if np.isneginf(l).all():
        return -1, 0.0
    if np.isposinf(l).any():
        l = np.where(np.isposinf(l), 0.0, -np.inf)
    V, m = len(l), l.max()
    if not t > 0:
        return int(np.argmax(l)), 1.0
    w = np.exp((l - m) / np.float64(t))
    w[np.isneginf(l)] = 0
    order = np.argsort(-l, kind="stable")
    n = V
    if 0 < top_k < V:
        n = int(top_k)
    if top_p < 1:
        c = np.cumsum(w[order[:n]])
        n = int(np.count_nonzero(c < np.float64(top_p) * c[-1])) + 1
    if min_p > 0:
        n = min(n, int(np.count_nonzero(w >= min(1.0, np.float64(min_p)))))
    keep = np.sort(order[:max(1, n)])
    c = np.cumsum(w[keep])
    u = 0.0 if not u > 0 else min(float(u), 1 - 2.0 ** -24)
    # a kept token of weight zero is never the first whose sum exceeds
    i = int(np.count_nonzero(c <= u * c[-1]))
    return int(keep[i]), float(w[keep[i]] / c[-1])


def _want(logits, u, t=None, top_k=None, top_p=None, min_p=None):
    l = logits.float().cpu().numpy()
    col = lambda v, d: [d] * len(l) if v is None else v.cpu().numpy()  # noqa: E731
    rows = [_one(*a) for a in zip(l, u.cpu().numpy(), col(t, 1.0), col(top_k, 0), col(top_p, 1.0), col(min_p, 0.0))]
    return np.array([r[0] for r in rows]), np.array([r[1] for r in rows])


def _run(nslm, logits, u, t=None, top_k=None, top_p=None, min_p=None, V=None):
    B = logits.shape[0]
    V = V or logits.shape[1]
    token = guard.buffer(B, torch.int32, fill=-7)
    prob = guard.buffer(B, torch.float32, fill=float("nan"))
    kind = nslm.NSLM_TYPE_BF16 if logits.dtype == torch.bfloat16 else nslm.NSLM_TYPE_F32
    p = None if t is top_k is top_p is min_p is None else nslm.sample_params(t, top_k, top_p, min_p)
    nslm.nslm_sample(logits, kind, B, V, logits.stride(0), p, u, token, prob)
    assert nslm.nslm_last_launch_count() == 1
    return token.cpu().numpy(), prob.cpu().numpy()


def _check(nslm, logits, u, **kw):
    token, prob = _run(nslm, logits, u, **kw)
    V = kw.pop("V", None)
    wt, wp = _want(logits[:, :V], u, **kw)
    assert np.array_equal(token, wt), np.flatnonzero(token != wt)
    assert np.all(np.abs(prob - wp) <= (2.0 ** -24 + 2.0 ** -29) * wp)


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _full(B, v, dtype=torch.float32):
    return torch.full((B,), v, dtype=dtype, device="cuda")


def _logits(B, V, seed, spread=3.0, dtype=torch.float32):
    return (spread * torch.randn(B, V, generator=_gen(seed), device="cuda")).to(dtype)


SIZES = [(1, 1), (3, 2), (2, 31), (4, 64), (5, 100), (33, 257), (7, 1000), (2, 4097), (3, 32003), (9, 50257),
         (2, 131072), (1, 262144), (200, 1500), (300, 33)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,V", SIZES)
def test_filters(nslm, B, V, dtype):
    u = torch.rand(B, generator=_gen(V), device="cuda")
    t = 0.5 + torch.rand(B, generator=_gen(V + 1), device="cuda")
    ks = torch.randint(1, V + 2, (B,), generator=_gen(V + 2), device="cuda").to(torch.int32)
    few = torch.randint(1, 60, (B,), generator=_gen(V + 5), device="cuda").to(torch.int32)
    ps = torch.rand(B, generator=_gen(V + 3), device="cuda")
    ms = 0.3 * torch.rand(B, generator=_gen(V + 4), device="cuda")
    # spread 0.1: nearly even, thousands of tokens kept; 0: all equal
    for spread in (3.0, 0.1, 0.0):
        l = _logits(B, V, V, spread, dtype)
        _check(nslm, l, u)
        _check(nslm, l, u, t=t)
        _check(nslm, l, u, t=t, top_k=ks)
        _check(nslm, l, u, top_k=few)
        _check(nslm, l, u, t=t, top_p=ps)
        _check(nslm, l, u, t=t, min_p=ms)
        _check(nslm, l, u, t=t, top_k=few, top_p=ps, min_p=ms)
        _check(nslm, l, u, t=t, top_k=ks, top_p=ps)


def test_many_random_numbers_on_one_row(nslm):
    # every token of a small row comes out where its interval lies
    V, B = 37, 1000
    l = _logits(1, V, 3, 2.0).expand(B, V).contiguous()
    u = (torch.arange(B, device="cuda") + 0.5) / B
    _check(nslm, l, u)
    _check(nslm, l, u, top_p=_full(B, 0.8))
    _check(nslm, l, u, top_k=_full(B, 5, torch.int32))


@pytest.mark.parametrize("V", [5, 64, 4099, 140000])
def test_ties(nslm, V):
    # equal logits: the first ones stay, and a random number picks by its size alone
    B = 64
    l = torch.zeros(B, V, device="cuda")
    u = torch.arange(B, device="cuda") / B
    token, prob = _run(nslm, l, u)
    assert np.array_equal(token, np.arange(B) * V // B)
    for k in (1, 2, V // 2, V - 1, V, V + 1):
        token, prob = _run(nslm, l, u, top_k=_full(B, k, torch.int32))
        n = V if k < 1 else min(k, V)
        assert np.array_equal(token, np.arange(B) * n // B), k
        assert np.all(prob == np.float32(1 / n))
    token, prob = _run(nslm, l, u, top_p=_full(B, 0.5))
    n = (V + 1) // 2
    assert np.array_equal(token, np.arange(B) * n // B)
    # two values, the threshold inside the lower one
    l[:, ::3] = 1.0
    high = (V + 2) // 3
    for k in (high, high + 1, V - 1):
        _check(nslm, l, u, top_k=_full(B, k, torch.int32), top_p=_full(B, 0.97))


def test_settings_at_and_past_their_ends(nslm):
    V = 500
    base = _logits(1, V, 9)
    nan, inf = float("nan"), float("inf")
    rows = []
    for t in (1.0, 0.0, -1.0, nan, 1e-30, 1e30, inf):
        rows += [dict(t=t), dict(t=t, top_k=3)]
    rows += [dict(top_k=v) for v in (-5, 0, 1, 2, V - 1, V, V + 1, 2**31 - 1, -2**31)]
    rows += [dict(top_p=v) for v in (-1.0, 0.0, 1e-30, 0.999999, 1.0, 2.0, nan, inf, -inf)]
    rows += [dict(min_p=v) for v in (-1.0, 0.0, 1e-30, 0.5, 1.0, 2.0, nan, inf, -inf)]
    rows += [dict(u=v) for v in (0.0, -1.0, nan, 1 - 2.0 ** -24, 1.0, 5.0, inf, -inf)]
    B = len(rows)
    l = base.expand(B, V).contiguous()
    col = lambda n, d, ty=torch.float32: torch.tensor([r.get(n, d) for r in rows], dtype=ty, device="cuda")  # noqa: E731
    kw = dict(t=col("t", 1.0), top_k=col("top_k", 0, torch.int32), top_p=col("top_p", 1.0), min_p=col("min_p", 0.0))
    u = col("u", 0.4)
    token, prob = _run(nslm, l, u, **kw)
    host = base[0].cpu().numpy()
    for i, r in enumerate(rows):
        a = dict(r)
        uu = a.pop("u", 0.4)
        if "u" in r and uu >= 1:  # just below 1: the last token with a weight
            want = int(np.flatnonzero(np.exp(host.astype(np.float64) - host.max()) > 2.0 ** -45)[-1])
            assert token[i] == want, r
            continue
        if "top_p" in a and not a["top_p"] < 1:
            a.pop("top_p")
        a = {n: np.float32(v) if n != "top_k" else v for n, v in a.items()}
        want, p = _one(host, np.float32(uu), **a)
        assert token[i] == want and abs(prob[i] - p) <= (2.0 ** -24 + 2.0 ** -29) * p, (r, token[i], want, prob[i], p)


def test_masked_logits(nslm):
    V, B = 3001, 12
    l = _logits(B, V, 4)
    inf, nan = float("inf"), float("nan")
    l[0] = -inf                                     # nothing left
    l[1] = nan
    l[2, :] = -inf
    l[2, V - 1] = -3.0                              # one left, the last
    l[3, ::2] = -inf
    l[4, ::2] = nan
    l[5, 1700] = inf                                # +inf alone
    l[6, [3, 1000, 2999]] = inf
    l[7, 100:] = torch.finfo(torch.float32).min     # masked by the type's lowest value
    l[8] = torch.finfo(torch.float32).min           # a row of nothing but those: all equal
    l[9] = torch.finfo(torch.float32).max
    l[10, 0] = nan
    l[10, 1:] = -inf
    l[11] *= 1e30                                   # far apart
    u = torch.rand(B, generator=_gen(8), device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        x = l.to(dtype)
        if dtype == torch.bfloat16:
            x[7, 100:] = torch.finfo(dtype).min
            x[8] = torch.finfo(dtype).min
            x[9] = torch.finfo(dtype).max
        _check(nslm, x, u)
        _check(nslm, x, u, top_k=_full(B, 40, torch.int32), top_p=_full(B, 0.9), min_p=_full(B, 0.01))
        _check(nslm, x, u, t=_full(B, 0.0))
        _check(nslm, x, u, top_p=_full(B, 0.3))


@pytest.mark.parametrize("V", [1, 37, 1001, 70001])
def test_rows_with_a_stride(nslm, V):
    # rows further apart than they are long, starting at odd addresses; what lies between is not looked at
    B, ld = 6, V + 13
    for dtype in (torch.float32, torch.bfloat16):
        whole = torch.full((B, ld), 1e4, device="cuda", dtype=dtype)
        whole[:, :V] = _logits(B, V, V, 2.0, dtype)
        u = torch.rand(B, generator=_gen(1), device="cuda")
        _check(nslm, whole, u, V=V)
        _check(nslm, whole, u, V=V, top_k=_full(B, 20, torch.int32), top_p=_full(B, 0.9))


def test_clustered_values(nslm):
    # values that differ by single steps of fp32, or that sit in two far clusters: the threshold search has to part them
    V, B = 20000, 4
    u = torch.rand(B, generator=_gen(2), device="cuda")
    step = (torch.randint(0, 3000, (B, V), generator=_gen(3), device="cuda").int() + 0x41200000).view(torch.float32)
    tiny = _logits(B, V, 5) * 1e-42                  # subnormal differences
    two = torch.where(_logits(B, V, 6) > 0, 5.0 + 1e-6 * _logits(B, V, 7), -20 + 1e-5 * _logits(B, V, 8))
    for l in (step, tiny, two):
        for k in (1, 7, 600, 5000, 19999):
            _check(nslm, l, u, top_k=_full(B, k, torch.int32))
        for p in (0.01, 0.5, 0.999):
            _check(nslm, l, u, top_p=_full(B, p))
            _check(nslm, l, u, top_k=_full(B, 9000, torch.int32), top_p=_full(B, p))


def test_optional_prob_captured_replayed_and_no_rows(nslm):
    B, V = 5, 5000
    l = _logits(B, V, 1)
    u = torch.rand(B, generator=_gen(1), device="cuda")
    k, p = _full(B, 30, torch.int32), _full(B, 0.9)
    token = guard.buffer(B, torch.int32, fill=-7)
    params = nslm.sample_params(None, k, p, None)
    nslm.nslm_sample(l, nslm.NSLM_TYPE_F32, B, V, V, params, u, token)
    assert np.array_equal(token.cpu().numpy(), _want(l, u, top_k=k, top_p=p)[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nslm.nslm_sample(l, nslm.NSLM_TYPE_F32, B, V, V, params, u, token)
    for seed in (5, 6):
        l.copy_(_logits(B, V, seed))
        u.copy_(torch.rand(B, generator=_gen(seed), device="cuda"))
        g.replay()
        assert np.array_equal(token.cpu().numpy(), _want(l, u, top_k=k, top_p=p)[0])
    token.fill_(-7)
    nslm.nslm_sample(l, nslm.NSLM_TYPE_F32, 0, V, V, params, u, token)
    assert nslm.nslm_last_launch_count() == 0 and bool((token == -7).all())


def test_offsets_past_32_bits(nslm):
    B, V, ld = 20, 1000, 1 << 27
    whole = torch.zeros(B, ld, dtype=torch.bfloat16, device="cuda")  # 5.4 GB
    whole[:, :V] = _logits(B, V, 3, 3.0, torch.bfloat16)
    u = torch.rand(B, generator=_gen(1), device="cuda")
    _check(nslm, whole, u, V=V, top_p=_full(B, 0.9))


# more rows than fit on the GPU at once: with one CTA a row, with two and more
LARGE = [(310, 3001), (310, 40001), (100, 60001), (70, 131072), (40, 262143)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,V", LARGE)
def test_large_batches(nslm, B, V, dtype):
    # rows at odd addresses, some with masked logits, some with nothing left
    ld = V + 3
    whole = torch.full((B, ld), 1e4, device="cuda", dtype=dtype)
    l = whole[:, :V]
    l.copy_(_logits(B, V, V, 3.0, dtype))
    inf = float("inf")
    l[5::17, ::2] = -inf
    l[6::17, 1::3] = float("nan")
    l[7] = -inf
    l[8, V // 2:] = torch.finfo(dtype).min
    l[9, [1, V // 3, V - 1]] = inf
    l[10] = 0.0
    l[11::17, :] *= 0.02                            # nearly even: the threshold is far down
    l[12, :] = -inf
    l[12, V - 1] = -2.0
    u = torch.rand(B, generator=_gen(V), device="cuda")
    t = 0.5 + torch.rand(B, generator=_gen(V + 1), device="cuda")
    t[::31] = 0
    ks = torch.randint(1, 3000, (B,), generator=_gen(V + 2), device="cuda").to(torch.int32)
    few = torch.randint(1, 60, (B,), generator=_gen(V + 5), device="cuda").to(torch.int32)
    ps = torch.rand(B, generator=_gen(V + 3), device="cuda")
    ms = 0.3 * torch.rand(B, generator=_gen(V + 4), device="cuda")
    _check(nslm, whole, u, V=V)
    _check(nslm, whole, u, V=V, t=t, top_k=few, top_p=ps, min_p=ms)
    _check(nslm, whole, u, V=V, t=t, top_k=ks, top_p=ps)
    _check(nslm, whole, u, V=V, top_p=ps)


def test_a_row_alone_and_in_a_large_batch_are_equal(nslm):
    # a row's draw does not depend on how many rows are drawn with it
    B, V = 80, 50257
    l = _logits(B, V, 17, 2.0)
    u = torch.rand(B, generator=_gen(3), device="cuda")
    for kw in (dict(), dict(top_k=_full(B, 50, torch.int32)), dict(top_p=_full(B, 0.9))):
        token, prob = _run(nslm, l, u, **kw)
        for i in (0, 41, 79):
            one = {n: v[:1] for n, v in kw.items()}
            a, b = _run(nslm, l[i:i + 1].clone(), u[i:i + 1].clone(), **one)
            assert a[0] == token[i] and b[0] == prob[i]


def test_two_calls_at_once(nslm):
    B, V = 48, 100000
    l = _logits(B, V, 23, 2.0)
    u = [torch.rand(B, generator=_gen(i), device="cuda") for i in range(2)]
    p = _full(B, 0.9)
    params = nslm.sample_params(None, None, p, None)
    out = [guard.buffer(B, torch.int32, fill=-7) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            nslm.nslm_sample(l, nslm.NSLM_TYPE_F32, B, V, V, params, u[i], out[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert np.array_equal(out[i].cpu().numpy(), _want(l, u[i], top_p=p)[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,V", [(6, 300), (6, 1025), (6, 5003), (6, 40000), (100, 20011)])
def test_lists_of_hundreds(nslm, B, V, dtype):
    # top-k from tens to past a thousand, over rows of one far outlier, of few values, and nearly even ones,
    # from cold to hot
    l = _logits(B, V, V + 1, 2.0, dtype)
    l[1::6, V // 3] = 900.0
    l[2::6] = (2 * l[2::6].float()).round().to(dtype) / 2
    l[3::6] *= 0.01
    l[4::6, : V // 2] = -float("inf")
    u = torch.rand(B, generator=_gen(V), device="cuda")
    for k in (60, 97, 250, 500, 1000, 1024, 1025):
        ks = _full(B, k, torch.int32)
        for t in (0.05, 1.0, 5.0):
            _check(nslm, l, u, t=_full(B, t), top_k=ks)
        _check(nslm, l, u, top_k=ks, top_p=_full(B, 0.95), min_p=_full(B, 0.001))


def test_thousands_of_infinite_logits_and_settings_left_out(nslm):
    B, V = 4, 20000
    l = _logits(B, V, 31)
    l[0, ::4] = float("inf")                        # more than a list holds
    l[1, :900] = float("inf")
    l[2, 3:] = -float("inf")
    u = torch.rand(B, generator=_gen(6), device="cuda")
    _check(nslm, l, u)
    for k in (2, 500, 2000, 7000):
        _check(nslm, l, u, top_k=_full(B, k, torch.int32))
        _check(nslm, l, u, top_k=_full(B, k, torch.int32), top_p=_full(B, 0.5))
    _check(nslm, l, u, top_p=_full(B, 0.25), min_p=_full(B, 0.5))
    # a struct of no arrays is no struct
    token = guard.buffer(B, torch.int32, fill=-7)
    nslm.nslm_sample(l, nslm.NSLM_TYPE_F32, B, V, V, nslm.sample_params(), u, token)
    assert np.array_equal(token.cpu().numpy(), _want(l, u)[0])
