"""GPU checks of the chunk attention's softmax weights where one position
outweighs the others: long contexts whose small weights add up, and scores of
any size that fp16 inputs reach.

The inputs are such that the result follows from a closed form in fp64: keys
of two kinds, so every row has two different scores.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from paged_kv_cache_152_gb300 import build
    build.build()
    import paged_kv_cache_152_gb300 as m
    m.load()
    return m


def run(pkv, q, keys, values, scale, num_ctas=0, bs=128, seed=0):
    """One sequence, one KV head; q [n][group][D], keys and values [L][D] on the GPU."""
    length, d = keys.shape
    blocks = -(-length // bs)
    order = torch.from_numpy(np.random.default_rng(seed).permutation(blocks + 1)[:blocks]).cuda()
    pools = []
    for rows in (keys, values):
        pool = torch.full((blocks + 1, 1, bs, d), float("nan"), dtype=torch.float16, device="cuda")
        padded = torch.full((blocks * bs, d), float("nan"), dtype=torch.float16, device="cuda")
        padded[:length] = rows
        pool[order, 0] = padded.view(blocks, bs, d)
        pools.append(pool)
    out = torch.full_like(q, -77.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.paged_attention_chunk(out, q, *pools, order[None].int(),
                              torch.tensor([length], dtype=torch.int32, device="cuda"),
                              torch.tensor([0, q.shape[0]], dtype=torch.int32, device="cuda"), scale,
                              num_ctas=num_ctas, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out.double().cpu().numpy()


def two_kinds(values, special, at, n, score):
    """fp64: row i of the last n of L positions sees positions up to L - n + i;
    position `at` (value `special`) has a score larger than the others' by
    `score`.  -> (out, spread) [n][D]; spread is sum_t softmax_t |v_t|."""
    length = values.shape[0]
    out, spread = [], []
    sums, mags = np.cumsum(values, axis=0), np.cumsum(np.abs(values), axis=0)
    for i in range(n):
        last = length - n + i
        rest, mag, count = sums[last], mags[last], last + 1
        w = 0.0
        if at <= last:
            w, count = 1.0, count - 1
            rest, mag = rest - values[at], mag - np.abs(values[at])
        small = np.exp(-score) if w else 1.0
        total = w + small * count
        out.append((w * special + small * rest) / total)
        spread.append((w * np.abs(special) + small * mag) / total)
    return np.stack(out), np.stack(spread)


@pytest.mark.parametrize("length,n,num_ctas", [(131072, 1, 1), (131072, 1, 2), (131072, 3, 0), (131072, 200, 4),
                                               (1 << 20, 1, 5), (1 << 20, 130, 0)])
@pytest.mark.parametrize("d", [64, 128])
def test_one_position_above_a_long_context(pkv, length, n, num_ctas, d):
    """An attention sink: one position about 17.5 above all others, which
    together still weigh length * e^-17.5.

    Tolerance: the output's rounding, 2^-11 |out| + 2^-25; a weight's rounding,
    2^-11 of it, or 2^-25 where it is below fp16's normal range.  The weights
    are placed at 2^9 and more for the row's maximum, so their sum is at
    least 2^9: the latter is at most 2^-34 of it for each position, whose
    values are at most 1.25.  The products' sums are fp32, cut at 2^-22 of the
    running sum at worst for each 16 positions that a CTA adds up; scores here
    have one term, exponent and ex2 2^-20, twice (numerator and sum); sums and
    joins 2^-14."""
    rng = np.random.default_rng(length + n)
    scale = d ** -0.5
    at = 777
    q = torch.zeros(n, 1, d, dtype=torch.float16, device="cuda")
    q[..., 3] = 1.0 / scale if d == 64 else 11.3125
    keys = torch.zeros(length, d, dtype=torch.float16, device="cuda")
    keys[at, 3] = 17.5
    score = scale * float(q[0, 0, 3]) * 17.5
    values = (1.0 + 0.25 * rng.random((length, d))).astype(np.float16)
    special = np.where(np.arange(d) % 2, 0.0, 0.75)
    values[at] = special
    got = run(pkv, q, keys, torch.from_numpy(values).cuda(), scale, num_ctas)[:, 0]
    values = values.astype(np.float64)
    ref, spread = two_kinds(values, special, at, n, score)
    ctas = num_ctas or torch.cuda.get_device_properties(0).multi_processor_count
    adds = length / min(ctas, length / 128) / 16
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (2.0 ** -11 + 2.0 ** -14 + 2.0 ** -18 + adds * 2.0 ** -22) * spread + \
        length * 2.0 ** -34 * 1.25
    over = np.abs(got - ref) / tol
    assert over.max() <= 1.0, over.max()


@pytest.mark.parametrize("a,b", [(1.0, 1.0), (30.0, 1000.0), (1000.0, 1000.0), (65504.0, 1000.0), (65504.0, 65504.0)])
@pytest.mark.parametrize("length,n,num_ctas", [(1, 1, 0), (300, 130, 0), (300, 200, 2), (1000, 1, 0), (1000, 1, 1),
                                               (700, 3, 1)])
def test_scores_of_any_size(pkv, a, b, length, n, num_ctas):
    """All keys the same but one: its rows return that position's value (or,
    for small scores, the mean that the scores give), the others the plain
    mean, however large the scores are.

    Tolerance: as above; equal scores are equal in fp32 too, and the two
    differ by 0.6 (one term; exponent's rounding 2^-20, twice) or by more
    than 1e5, where the smaller weights are zero in any arithmetic."""
    d, scale = 128, 0.3
    rng = np.random.default_rng(length + n)
    at = max(0, length - n // 2 - 1)
    one = b == 1.0
    q = torch.zeros(n, 2, d, dtype=torch.float16, device="cuda")
    keys = torch.zeros(length, d, dtype=torch.float16, device="cuda")
    width = 1 if one else d
    q[..., :width] = a
    keys[:, :width] = -b
    keys[at, :width] = b
    score = 2 * float(np.float32(scale)) * a * b * width
    values = rng.standard_normal((length, d)).astype(np.float16)
    got = run(pkv, q, keys, torch.from_numpy(values).cuda(), scale, num_ctas, bs=16)
    values = values.astype(np.float64)
    ref, spread = two_kinds(values, values[at], at, n, score)
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (2.0 ** -11 + 2.0 ** -14 + 2.0 ** -18) * spread + length * 2.0 ** -34 * 5.5
    for h in range(2):
        over = np.abs(got[:, h] - ref) / tol
        assert over.max() <= 1.0, over.max()
