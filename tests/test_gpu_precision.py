"""How exact the shared-prefix and scored attention are where a rule of their kernels says so.

The tensor cores add in fp32 and cut each sum to 24 bits toward zero: a product's sum loses less than 2^-23 of itself, so N
products in a row that add values of one sign lose less than N / 2 * 2^-23 of the result (the sums grow evenly).  With queries
of zeros every score is 0 and every weight exactly 1, and what is left is that, and some fp32 roundings of 2^-24 each."""
import math

import pytest
import torch

import looped_lm_decode_b200 as LQ
from tests.test_gpu_edges import bf16, gen, i32

pytestmark = pytest.mark.gpu

CUT = 2.0 ** -23


def positive(g, *shape):
    """Of many magnitudes: sums of many of them need more than 24 bits."""
    return torch.randn(*shape, generator=g, device="cuda").exp().bfloat16()


def off(out, v):
    """The largest relative error of out [rows][Hq][D] against the means of v [Hkv][n][D]."""
    want = v.double().mean(1).repeat_interleave(out.shape[1] // v.shape[0], 0)
    return ((out.double() - want) / want).abs().max().item()


@pytest.mark.parametrize("n,rows,hkv,hq,d", [(32768, 2048, 16, 16, 128), (32768, 200, 16, 16, 128), (30001, 600, 40, 40, 64),
                                             (70001, 40, 40, 40, 64), (131072, 64, 4, 16, 128)])
def test_rows_as_m_do_not_drift_over_long_prefixes(n, rows, hkv, hq, d):
    """At most 4096 tokens, 256 products of weights with a remainder of 0, in a run; then sums of at most 32 runs and some
    twenty roundings of the merge and the division.  (Without runs 2048 products in the largest cases.)"""
    g = gen(n + rows)
    k, v = bf16(g, 1, hkv, n, d), positive(g, 1, hkv, n, d)
    out, lse = LQ.bf16_shared_attn(LQ.Bf16Cache(k, v, hq), 0, torch.zeros(rows, hq, d, dtype=torch.bfloat16, device="cuda"), i32([n]), n)
    LQ.fault_check()
    assert off(out, v[0]) <= 256 / 2 * CUT + (32 + 20) * 2.0 ** -24
    assert (lse - math.log(n)).abs().max().item() <= 2.0 ** -23 * math.log(n) + 1e-5


def test_runs_with_a_rising_maximum_and_an_other_part():
    """Sums of runs follow the maximum: scores that rise by 2^8 and more from run to run, and fall again."""
    g, n, rows, d = gen(2), 32768, 2000, 64
    k, v, q = bf16(g, 1, 16, n, d), bf16(g, 1, 16, n, d), bf16(g, rows, 16, d)
    q[..., 0] = 8
    t = torch.linspace(-1, 1, n, device="cuda")
    k[0, :, :, 0] = (40 * torch.where(t < 0.4, t, 0.8 - t)).bfloat16()
    other = torch.randn(rows, 16, d, generator=g, device="cuda"), 10 + torch.randn(rows, 16, generator=g, device="cuda")
    for o in (None, other):
        out, lse = LQ.bf16_shared_attn(LQ.Bf16Cache(k, v, 16), 0, q, i32([n]), n, other=o)
        LQ.fault_check()
        for r, h in ((0, 0), (777, 7), (1999, 15)):
            s = k[0, h].double() @ q[r, h].double() / math.sqrt(d)
            l = torch.logsumexp(s, 0)
            joint = l if o is None else torch.logaddexp(l, o[1][r, h].double())
            p = torch.exp(s - joint)
            want, mag = p @ v[0, h].double(), p @ v[0, h].double().abs()
            if o is not None:
                po = torch.exp(o[1][r, h].double() - joint)
                want, mag = want + po * o[0][r, h].double(), mag + po * o[0][r, h].double().abs()
            # |q k| scale reaches 48: test_gpu_shared.py's bounds for sums below 8, times 7
            assert ((out[r, h].double() - want).abs() <= 7 * 2.5e-4 * mag).all()
            assert abs(lse[r, h].item() - joint.item()) <= 7e-4


def test_an_other_part_in_place_with_runs():
    g, n, rows, d = gen(3), 32768, 2000, 64
    k, v, q = bf16(g, 1, 16, n, d), bf16(g, 1, 16, n, d), bf16(g, rows, 16, d)
    cache, lens = LQ.Bf16Cache(k, v, 16), i32([n])
    other = torch.randn(rows, 16, d, generator=g, device="cuda"), 10 + torch.randn(rows, 16, generator=g, device="cuda")
    want = LQ.bf16_shared_attn(cache, 0, q, lens, n, other=other)
    again = LQ.bf16_shared_attn(cache, 0, q, lens, n, other=other)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
    out = other[0].clone()
    LQ.bf16_shared_attn(cache, 0, q, lens, n, other=(out, other[1]), out=out)
    assert torch.equal(out, want[0])


@pytest.mark.parametrize("n,rows,hkv,hq,d", [(32768, 8, 148, 148, 64), (131072, 3, 16, 32, 128), (32768, 30, 148, 148, 64)])
def test_tokens_as_m_move_o_every_fourth_tile(n, rows, hkv, hq, d):
    """32 products in a run; then at most 32 moves, 40 records and 20 roundings.  (Without the moves 1024 products in the
    largest cases.)"""
    g = gen(n + rows)
    k, v = bf16(g, 1, hkv, n, d), positive(g, 1, hkv, n, d)
    out, _ = LQ.bf16_shared_attn(LQ.Bf16Cache(k, v, hq), 0, torch.zeros(rows, hq, d, dtype=torch.bfloat16, device="cuda"), i32([n]), n)
    LQ.fault_check()
    assert off(out, v[0]) <= 32 / 2 * CUT + (32 + 40 + 20) * 2.0 ** -24


def test_scored_decode_on_the_tensor_cores_moves_o_every_fourth_tile():
    g, b, n, hkv, hq, d = gen(5), 10, 32768, 16, 32, 64
    k, v = bf16(g, b, hkv, n, d), positive(g, b, hkv, n, d)
    q = torch.zeros(b, hq, d, dtype=torch.bfloat16, device="cuda")
    out, lse, score = LQ.bf16_decode_attn_scored(LQ.Bf16Cache(k, v, hq), q, i32([n] * b), n, None,
                                                 score_out=torch.zeros(b, hkv, n, device="cuda"))
    LQ.fault_check()
    for i in range(b):
        assert off(out[i:i + 1], v[i]) <= 32 / 2 * CUT + (32 + 4 + 20) * 2.0 ** -24
    # two heads of weights 1 / n; the log-sum-exp is 15 log2 units and holds them to 15 * 2^-24 and the roundings of exp2 and log2
    assert (score * n / 2 - 1).abs().max().item() <= 2.0 ** -19


@pytest.mark.parametrize("rows,hkv,hq,d", [(1, 1, 1, 128), (5, 2, 8, 64), (32, 4, 4, 128), (40, 4, 4, 128), (100, 2, 4, 64)])
@pytest.mark.parametrize("n", [2, 30, 300])
def test_weights_of_short_calls_are_held_in_fp32(n, rows, hkv, hq, d):
    """One token of value 1 among tokens of value 0: the output is its weight p / sum.  Its score is one product, exact;
    the exponent's factor is off by 2^-23 of at most 1.02 (5.2 at 300 tokens' worth), exp2 by 2^-22.5, and some six
    roundings follow.  A weight in two bf16 parts would be off by up to 2^-17."""
    g = gen(n + rows)
    k, v = torch.zeros(1, hkv, n, d, device="cuda").bfloat16(), torch.zeros(1, hkv, n, d, device="cuda").bfloat16()
    at = n // 2
    k[0, :, at, 0], v[0, :, at] = 1, 1
    q = bf16(g, rows, hq, d)
    q[..., 0] = -8 * torch.rand(rows, hq, generator=g, device="cuda")
    out, lse = LQ.bf16_shared_attn(LQ.Bf16Cache(k, v, hq), 0, q, i32([n]), n)
    LQ.fault_check()
    s = q[..., 0].double() / math.sqrt(d)
    want = torch.exp(s) / (torch.exp(s) + n - 1)
    assert ((out.double() / want[..., None]) - 1).abs().max().item() <= 1.1 * 2.0 ** -22.5 + 8 * 2.0 ** -24
    assert (lse.double() - torch.log(torch.exp(s) + n - 1)).abs().max().item() <= 1e-6


@pytest.mark.parametrize("rows,n", [(3, 2), (3, 52), (3, 500), (60, 2), (60, 52), (60, 250), (200, 52)])
def test_rebuilt_keys_of_short_calls_are_held_in_fp32(rows, n):
    """Queries of one channel, 64: a score is 64 / sqrt(D) = 8 times one channel of a rotated key of up to 4.  The rotation's two
    roundings, its table's and the sums of its parts leave 6 * 2^-24 of 32; two bf16 parts would leave 2^-17 of it, 2.4e-4."""
    from tests.test_gpu_shared import make_coded, rebuild
    g, hkv, d = gen(rows + n), 2, 64
    cache = make_coded(g, hkv, hkv, d, 4, 4, 1, 256, 1, (n + 3) // 4 * 4)
    q = torch.zeros(rows, hkv, d, device="cuda").bfloat16()
    for r in range(rows):
        q[r, :, (7 * r) % d] = 64
    out, lse = LQ.shared_attn(cache, 0, 1, 0, q, i32([n]), n)
    LQ.fault_check()
    k, v = rebuild(cache, 1, 0, 0, n)
    assert k.abs().max().item() < 8
    s = torch.einsum("rhd,hnd->rhn", q.double(), k) / math.sqrt(d)
    want, mag = torch.softmax(s, 2), 8 * k.abs().max().item()
    few = 6 * 2.0 ** -24 * mag + 16 * 2.0 ** -24
    assert (lse.double() - torch.logsumexp(s, 2)).abs().max().item() <= few + 2.0 ** -22 * torch.logsumexp(s, 2).abs().max().item()
    ref = torch.einsum("rhn,hnd->rhd", want, v)
    size = torch.einsum("rhn,hnd->rhd", want, v.abs())
    assert ((out.double() - ref).abs() <= (2 * few + 2e-6) * size).all()


@pytest.mark.parametrize("coded", [False, True])
def test_a_wait_that_runs_out_with_runs(coded):
    """Rows of NaN, a fault, and the next call as before, where O had left tensor memory, too."""
    from tests.test_gpu_edges import coded_cache
    g, n, rows, d = gen(6), 20000, 2000 if not coded else 600, 64
    q, lens = bf16(g, rows, 16, d), i32([n])
    if coded:
        cache = coded_cache(g, 16, 16, d, 4, 4, 256, n)
        call = lambda: LQ.shared_attn(cache, 0, 1, 0, q, lens, n)  # noqa: E731
    else:
        cache = LQ.Bf16Cache(bf16(g, 1, 16, n, d), bf16(g, 1, 16, n, d), 16)
        call = lambda: LQ.bf16_shared_attn(cache, 0, q, lens, n)  # noqa: E731
    good = call()
    LQ.fault_check()
    before = LQ.wait_limit_ns()
    LQ.set_wait_limit_ns(0)
    try:
        bad = call()
        with pytest.raises(LQ.LoopVQError) as e:
            LQ.fault_check()
        assert e.value.status == 5 and bad[0].isnan().all() and bad[1].isnan().all()
    finally:
        LQ.set_wait_limit_ns(before)
    again = call()
    LQ.fault_check()
    assert torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])
