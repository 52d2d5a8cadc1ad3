"""GPU: gqa_paged_attn over sequences so long that one block sums up hundreds of thousands of tokens, with and without a
window and sinks, against the plain 64-bit form (pages that stand in the block tables many times, as in
test_gpu_tree_long)."""
import math

import pytest
import torch

import gqa_attention_kv_split_gb300 as gqa
from test_gpu_tree_long import BF16, DEV, E4M3, F16, LONG, PAGE, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    gqa.build()
    yield
    assert gqa.gqa_check_device_errors(0) == 0


def counts(table, lo, hi, num):
    """How often each place of the pages stands between the tokens lo and hi of a sequence."""
    f = torch.zeros(num, PAGE, dtype=torch.float64)
    for end, sign in ((hi, 1), (lo, -1)):
        f += sign * torch.bincount(table[:end // PAGE].long(), minlength=num)[:, None]
        if end % PAGE:
            f[int(table[end // PAGE]), :end % PAGE] += sign
    return f


def plain(q, k, v, table, lens, window, sinks, rows):
    hq, d, hkv = q.shape[1], q.shape[2], k.shape[1]
    ks, vs = (x.double().permute(1, 0, 2, 3).reshape(hkv, -1, d).repeat_interleave(hq // hkv, 0) for x in (k, v))
    out, lse, mag, reach = [], [], [], []
    for b in rows:
        first = max(0, lens[b] - window) if window else 0
        f = counts(table[b], first, lens[b], k.shape[0]) + counts(table[b], 0, min(sinks, first), k.shape[0])
        s = torch.einsum("hd,hnd->hn", q[b].double(), ks) / math.sqrt(d) + f.view(-1).log()
        lse.append(torch.logsumexp(s, -1))
        p = torch.exp(s - lse[-1][:, None])
        out.append(torch.einsum("hn,hnd->hd", p, vs))
        mag.append(torch.einsum("hn,hnd->hd", p, vs.abs()))
        reach.append(torch.einsum("hd,hnd->hn", q[b].double().abs(), ks.abs()).amax(-1) / math.sqrt(d))
    return (torch.stack(x) for x in (out, lse, mag, reach))


def check(lens, hq, hkv, d, dtype, cache, window=0, sinks=0, rising=False, seed=0):
    """The bound: half a step of the output; a weight's two terms and the scores' error as in paged_reference; the
    product with V, whose accumulators take two sums for 16 tokens, each off by 2^-23 of what has been summed, for 8192
    tokens of a warp at most before they are added to a sum in f32, one rounding (2^-24) for 8192 tokens; and the sums of
    the weights, one addition (2^-24) a thread for 16 of its warp's tokens: 1 / 8 of all, 1 / 4 at head dim 256."""
    q, k, v, table = make(lens, 1, hq, hkv, d, dtype, cache, rising, seed)
    lse = torch.full((len(lens), hq), 9.0, device=DEV)
    got = gqa.gqa_paged_attn(q.to(DEV), k.to(DEV), v.to(DEV), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), lse=lse,
                             window=window, sinks=sinks)
    torch.cuda.synchronize()
    rows = sorted({0, len(lens) // 2, len(lens) - 1})
    out, want_lse, mag, reach = plain(q, k, v, table, lens, window, sinks, rows)
    assert torch.isfinite(got).all()
    eps, own = torch.finfo(dtype).eps, max(lens) / (4 if d == 256 else 8)  # tokens of a warp
    s_err = 2.0 ** -19 * reach + 2.0 ** -20
    sums = 2.0 ** -23 * min(own, 8192) / 8 + 2.0 ** -24 * own / 8192
    weights = 2.0 ** -24 * (own / 16 + 64)
    tol = eps / 2 * out.abs() + (1 + eps) * (2.0 ** -16 + sums + weights + 2 * s_err)[..., None] * mag
    err = (got.cpu()[rows].double() - out).abs()
    assert (err <= tol).all(), f"out: worst {float((err / tol).max()):.2f} of the bound, {float((err / mag).max()):.2e} of sum p |v|"
    e = (lse.cpu()[rows].double() - want_lse).abs()
    assert (e <= s_err + weights + 2.0 ** -20 * want_lse.abs()).all()
    # What a long sum is off by does not go to one side.
    rel = ((got.cpu()[rows].double() - out) / out)[..., :d // 2]
    drift = abs(float(rel.mean()))
    assert drift <= eps / 2 / math.sqrt(rel.numel()) * 4 + 2.0 ** -17 + sums / 2, drift
    return got


TYPES = [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("hq", [32, 128])
def test_a_million_tokens_in_one_block(hq, dtype, cache, d):
    """4 and 16 heads a KV head."""
    check([LONG] * 19, hq, 8, d, dtype, cache, seed=d)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_under_a_window_with_sinks(dtype, cache, d):
    check([LONG - 1000 * i for i in range(19)], 32, 8, d, dtype, cache, window=700000, sinks=90000, seed=d)
    check([LONG] * 20, 24, 8, d, dtype, cache, window=600001, seed=d)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_maxima_that_rise_between_the_sums(dtype, cache, d):
    check([400000] * 19, 32, 8, d, dtype, cache, rising=True, seed=d)
    check([400000] * 19, 80, 8, d, dtype, cache, rising=True, seed=d)


@pytest.mark.parametrize("tokens", [65536, 65537, 65664, 131072, 131073, 196737])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cache", [F16, E4M3])
def test_around_the_sums_own_lengths(tokens, d, cache):
    check([tokens] * 20, 16, 8, d, F16, cache, seed=d)
    check([tokens // 2] * 20, 96, 8, d, F16, cache, seed=d)


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_pieces_and_several_units_of_a_block(cache, hkv):
    """Units that go through sums of their own after, and before, units that do not."""
    check([1000000, 500, 1400001, 800000, 123] * 5, 4 * hkv, hkv, 128, BF16, cache, seed=hkv)
    check([200000, 70000, 20, 300000] * 12, 16 * hkv, hkv, 64, BF16, cache, rising=True, seed=hkv)


def test_same_bits_every_time():
    want = check([900000] * 25, 32, 8, 128, F16, F16, seed=3)
    for _ in range(3):
        assert torch.equal(check([900000] * 25, 32, 8, 128, F16, F16, seed=3), want)
