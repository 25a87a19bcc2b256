"""nslm_q4_gemv against the product in 64 bits.

Two kinds of data.  Small integers with power-of-two scales, whose every
partial sum is an integer multiple of 1/4 below 2^22: fp32 holds all of them,
in any order of summation, so the result has to be equal.  And random ones,
held to the rounding of a sum: a group's terms are added first (at most G of
them), then the groups and the partial sums of a row (at most K / G + 32), each
addition off by at most 2^-23 of the sums of magnitudes (twice fp32's half
step, for sums that truncate)."""
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


def _weights(N, K, G, affine, seed, whole):
    g = torch.Generator("cuda").manual_seed(seed)
    q = torch.randint(-2**31, 2**31, (N, K // 8), generator=g, device="cuda", dtype=torch.int32)
    if whole:
        scales = 2.0 ** torch.randint(-1, 2, (N, K // G), generator=g, device="cuda")
        biases = torch.randint(-15, 16, (N, K // G), generator=g, device="cuda") / 2
    else:
        scales = 0.01 * torch.exp(torch.randn(N, K // G, generator=g, device="cuda"))
        biases = -7.5 * scales + 0.02 * torch.randn(N, K // G, generator=g, device="cuda")
    return q, scales.bfloat16(), biases.bfloat16() if affine else None


def _x(M, K, seed, whole):
    g = torch.Generator("cuda").manual_seed(seed)
    if whole:
        return torch.randint(-4, 5, (M, K), generator=g, device="cuda").bfloat16()
    return torch.randn(M, K, generator=g, device="cuda").bfloat16()


def _dense(q, scales, biases, G):
    """Weights, and their parts' magnitudes, in 64 bits."""
    shift = torch.arange(0, 32, 4, device=q.device, dtype=torch.int32)
    n = ((q.unsqueeze(-1) >> shift) & 15).double().reshape(q.shape[0], -1)
    s = scales.double().repeat_interleave(G, 1)
    b = biases.double().repeat_interleave(G, 1) if biases is not None else -8 * s
    return s * n + b, s.abs() * n + b.abs()


def _run(nslm, q, scales, biases, G, x, flags=0, stream=None):
    M = x.shape[0]
    y = guard.buffer((M, q.shape[0]), torch.float32, fill=float("nan"))
    nslm.nslm_q4_gemv(nslm.q4_matrix(q, scales, biases, G), x, M, y, flags, stream)
    assert nslm.nslm_last_launch_count() == 1
    return y


SHAPES = [(1, 32, 32), (1, 64, 64), (1, 128, 128), (3, 96, 32), (15, 160, 32), (16, 192, 64), (17, 384, 128),
          (33, 1408, 32), (100, 1408, 64), (100, 1408, 128), (257, 2048, 32), (512, 1024, 64), (65, 4096, 128),
          (31, 8192, 64), (2049, 640, 128), (9000, 256, 32), (40, 224, 32), (5, 65536, 32)]


@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("N,K,G", SHAPES)
def test_whole_numbers_are_equal(nslm, N, K, G, affine):
    q, scales, biases = _weights(N, K, G, affine, 11 * N + K, True)
    w, _ = _dense(q, scales, biases, G)
    for M in range(1, 9):
        if M * K > 65536:
            break
        x = _x(M, K, M, True)
        y = _run(nslm, q, scales, biases, G, x, flags=M & 1)
        assert torch.equal(y.double(), x.double() @ w.t()), M


# enough rows for a tile a warp (their scales come 16 bytes at once where K is a
# multiple of 8 groups), and rows so long that the activations take the room of
# a second CTA, or of most warps
LONG = [(40000, 512, 32, 1), (40001, 512, 64, 4), (38000, 1024, 128, 3), (39990, 1536, 64, 8), (40000, 1000 * 32, 32, 1),
        (33153, 8192, 32, 8), (35000, 8192, 64, 8), (33200, 8192, 128, 5), (120, 16384, 32, 4), (700, 32768, 64, 2),
        (19000, 16384, 64, 3), (2400, 65536, 128, 1), (37000, 7 * 256, 32, 6), (2500, 6000 // 32 * 32, 32, 7)]


@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("N,K,G,M", LONG)
def test_many_rows_and_long_ones_are_equal(nslm, N, K, G, M, affine):
    q, scales, biases = _weights(N, K, G, affine, N + K, True)
    x = _x(M, K, N, True)
    y = _run(nslm, q, scales, biases, G, x)
    for i in range(0, N, 4096):
        b = biases[i:i + 4096] if affine else None
        w, _ = _dense(q[i:i + 4096], scales[i:i + 4096], b, G)
        # any partial sum, however the offset is taken apart: halves below 2^22
        size = 16 * scales[i:i + 4096].double().repeat_interleave(G, 1)
        if affine:
            size += b.double().abs().repeat_interleave(G, 1)
        assert float((x.double().abs() @ size.t()).max()) < 2**22
        assert torch.equal(y[:, i:i + 4096].double(), x.double() @ w.t()), i


@pytest.mark.parametrize("N,K,G,M,affine", [(100, 1408, 128, 5, False), (512, 1024, 64, 1, True), (2048, 4096, 32, 1, True),
                                            (333, 8192, 64, 8, True), (1000, 2048, 32, 3, False), (64, 16384, 128, 4, True)])
def test_random_numbers_within_rounding(nslm, N, K, G, M, affine):
    q, scales, biases = _weights(N, K, G, affine, N + K, False)
    w, parts = _dense(q, scales, biases, G)
    x = _x(M, K, 5, False)
    y = _run(nslm, q, scales, biases, G, x).double()
    want = x.double() @ w.t()
    bound = (G + K // G + 32) * 2.0 ** -23 * (x.double().abs() @ parts.t())
    assert bool(((y - want).abs() <= bound).all())
    # over all rows the errors have no common sign: a walk of so many steps
    # instead of their sum
    walk = (G + K // G + 32) ** 0.5 * 2.0 ** -23 * torch.sqrt(x.double().square() @ parts.square().t())
    assert float((y - want).norm()) <= float(walk.norm())


def test_two_calls_give_equal_bits(nslm):
    q, scales, biases = _weights(5000, 2048, 64, True, 3, False)
    x = _x(8, 2048, 4, False)
    a = _run(nslm, q, scales, biases, 64, x)
    b = _run(nslm, q, scales, biases, 64, x, flags=nslm.NSLM_GEMV_FIELDS_READY)
    assert torch.equal(a, b)


def test_large_activations_and_zero_scales(nslm):
    # bf16's range is fp32's: a product near its top, and groups that are zero
    N, K, G = 48, 256, 32
    q, scales, biases = _weights(N, K, G, True, 9, True)
    scales[::3] = 0
    biases[::3] = 0
    w, _ = _dense(q, scales, biases, G)
    x = _x(2, K, 1, True) * 2.0 ** 100
    y = _run(nslm, q, scales, biases, G, x)
    assert torch.equal(y.double(), x.double() @ w.t())
    assert bool((y[:, ::3] == 0).all())


def test_rows_of_a_stack_and_of_a_larger_batch(nslm):
    # one expert's rows of stacked weights, and one chunk of a longer batch of vectors
    N, K, G = 96, 512, 64
    q, scales, biases = _weights(4 * N, K, G, True, 21, True)
    x = _x(13, K, 2, True)
    w, _ = _dense(q, scales, biases, G)
    y = _run(nslm, q[N:2 * N], scales[N:2 * N], biases[N:2 * N], G, x[4:12])
    assert torch.equal(y.double(), x[4:12].double() @ w[N:2 * N].t())


def test_offsets_past_32_bits(nslm):
    N, K, G = 1_060_000, 8192, 128  # 4.3 GB of nibbles
    q = torch.zeros(N, K // 8, dtype=torch.int32, device="cuda")
    scales = torch.ones(N, K // G, dtype=torch.bfloat16, device="cuda")
    last, s, _ = _weights(40, K, G, False, 1, True)
    q[-40:], scales[-40:] = last, s
    x = _x(1, K, 3, True)
    y = _run(nslm, q, scales, None, G, x)
    w, _ = _dense(last, s, None, G)
    assert torch.equal(y[0, -40:].double(), (x.double() @ w.t())[0])
    assert torch.equal(y[0, :-40].double(), (-8 * x.double().sum()).expand(N - 40))


def test_chain_on_a_side_stream_and_replayed(nslm):
    # products that feed one another (the early weight loads must not run
    # ahead of the activations), eager on a side stream and from a graph
    N, K, G = 512, 512, 64
    q, scales, biases = _weights(N, K, G, True, 31, True)
    w, _ = _dense(q, scales, biases, G)
    W = nslm.q4_matrix(q, scales, biases, G)
    x = guard.buffer((1, K), torch.bfloat16, fill=0)
    y = guard.buffer((1, N), torch.float32, fill=float("nan"))
    z = guard.buffer((1, N), torch.float32, fill=float("nan"))
    h = guard.buffer((1, K), torch.bfloat16, fill=0)

    def step():
        nslm.nslm_q4_gemv(W, x, 1, y, nslm.NSLM_GEMV_FIELDS_READY)
        h.copy_(y.clamp(-4, 4).round())
        nslm.nslm_q4_gemv(W, h, 1, z, nslm.NSLM_GEMV_FIELDS_READY)

    def want():
        a = (x.double() @ w.t()).float().clamp(-4, 4).round().bfloat16()
        return a.double() @ w.t()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x.copy_(_x(1, K, 50, True))
        step()
    s.synchronize()
    assert torch.equal(z.double(), want())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (51, 52):
        x.copy_(_x(1, K, seed, True))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(z.double(), want())


def test_no_rows(nslm):
    q = torch.zeros(16, 4, dtype=torch.int32, device="cuda")
    y = guard.buffer((1, 16), torch.float32, fill=7.0)
    W = nslm.nslm_q4_matrix(q.data_ptr(), q.data_ptr(), 0, 0, 32, 32)
    nslm.nslm_q4_gemv(W, q, 1, y)
    assert nslm.nslm_last_launch_count() == 0
    assert bool((y == 7).all()) and np.isfinite(float(y.sum()))


def test_two_calls_at_once(nslm):
    # two streams, two outputs, one matrix and one x: calls share nothing that they write
    N, K, G = 20000, 2048, 64
    q, scales, biases = _weights(N, K, G, True, 61, True)
    w, _ = _dense(q, scales, biases, G)
    x = _x(8, K, 3, True)
    want = x.double() @ w.t()
    W = nslm.q4_matrix(q, scales, biases, G)
    ys = [guard.buffer((8, N), torch.float32, fill=float("nan")) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, y in zip(streams, ys):
            nslm.nslm_q4_gemv(W, x, 8, y, nslm.NSLM_GEMV_FIELDS_READY, s)
    torch.cuda.synchronize()
    for y in ys:
        assert torch.equal(y.double(), want)
