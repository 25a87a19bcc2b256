"""nslm_q4_gemv at the ends of what it takes: the longest rows for each number of
vectors, where the activations leave the least shared memory.

Small integers with power-of-two scales: every partial sum is an integer
multiple of a power of two, below 2^22 of them, so fp32 holds it and the result
has to be equal."""
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


def _weights(N, K, G, affine, seed, exponent=0):
    g = torch.Generator("cuda").manual_seed(seed)
    q = torch.randint(-2**31, 2**31, (N, K // 8), generator=g, device="cuda", dtype=torch.int32)
    scales = 2.0 ** (torch.randint(0, 2, (N, K // G), generator=g, device="cuda") + exponent)
    biases = torch.randint(-15, 16, (N, K // G), generator=g, device="cuda") * 2.0 ** exponent
    return q, scales.bfloat16(), biases.bfloat16() if affine else None


def _dense(q, scales, biases, G):
    shift = torch.arange(0, 32, 4, device=q.device, dtype=torch.int32)
    n = ((q.unsqueeze(-1) >> shift) & 15).double().reshape(q.shape[0], -1)
    s = scales.double().repeat_interleave(G, 1)
    return s * n + biases.double().repeat_interleave(G, 1) if biases is not None else s * (n - 8)


@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8])
def test_the_longest_rows(nslm, M, G, affine):
    most = 65536 // (M if M <= 2 else 4 if M <= 4 else 8)
    for K in sorted({most, most - G, most * 15 // 16 // G * G}):
        for N in (3, 2500):
            q, scales, biases = _weights(N, K, G, affine, K + N)
            g = torch.Generator("cuda").manual_seed(M)
            x = torch.randint(-1, 2, (M, K), generator=g, device="cuda").bfloat16()
            y = guard.buffer((M, N), torch.float32, fill=float("nan"))
            nslm.nslm_q4_gemv(nslm.q4_matrix(q, scales, biases, G), x, M, y)
            # at most 2^16 terms of up to 46 (15 times 2, and 16 that an offset is taken apart by): below 2^22
            assert torch.equal(y.double(), x.double() @ _dense(q, scales, biases, G).t()), (K, N)


@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("G", [32, 64, 128])
def test_the_largest_activations(nslm, G, affine):
    # a group's sums before the scale reach 128 * 8 * 2^117 = 2^127; small scales bring the rows back
    N, K = 40, 1024
    q, scales, biases = _weights(N, K, G, affine, G, exponent=-40)
    g = torch.Generator("cuda").manual_seed(G)
    x = torch.randint(-1, 2, (3, K), generator=g, device="cuda")
    x[0], x[1] = 1, -1
    q[0] = 0                                         # every weight the lowest
    x = (x * 2.0 ** 100 * 2.0 ** 17).bfloat16()
    y = guard.buffer((3, N), torch.float32, fill=float("nan"))
    nslm.nslm_q4_gemv(nslm.q4_matrix(q, scales, biases, G), x, 3, y)
    assert bool(torch.isfinite(y).all())
    assert torch.equal(y.double(), x.double() @ _dense(q, scales, biases, G).t())
