"""GPU: what gqa_paged_attn keeps of its numbers, held to bounds that leave no room for
a shorter weight, a query element that has lost bits, or a cap that costs the score."""
import pytest
import torch

import gqa_attention_kv_split_gb300 as gqa
import paged_reference as R
from test_gpu_paged_attn import BF16, DEV, E4M3, F16, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    gqa.build()
    yield
    assert gqa.gqa_check_device_errors(0) == 0


def check(x, **kw):
    """As paged_reference.check_attention, with these two parts narrower.  A weight meets V as two terms:
    each is off by half a step, 2^-8 in bf16 (bf16 pages) and 2^-11 in f16, of what it has to hold, so that
    the pair is off by 2^-16 or 2^-22.  The cap c tanh(s / c) has a slope of 1 at most, so that it passes on
    the score's error.  Its own is relative: with |s / c| at 1/4 at least, tanh as 1 - 2 r, r = 1 / (e + 1),
    has from the exponential e (2^-22 of it), the sum (2^-24), the reciprocal (2^-23) and the exponent's
    roundings at most 1.6 * 2^-22, which is 2^-19 of tanh(1/4); nearer to 0 the series is off by less than
    2^-23.  So 2^-19 of the capped score, which is at most min(c, reach).  A bf16 query over E4M3 pages enters
    the product in f16, its row's largest element at 2^15 at least: f16's spacing is nowhere below 2^-24, so
    that an element is off by half of it, 2^-25, at most: 2^-40 of the largest one, times |k| in the score."""
    q = x[0]
    lse = torch.full(q.shape[:2], 9.0, device=DEV)
    got = gqa.gqa_paged_attn(*x, lse=lse, **kw).cpu()
    q, k, v, table, lens = (t.cpu() for t in x)
    out, want_lse, mag, reach = R.attention(q, k, v, table, lens, **kw)
    s_err = 2.0 ** -19 * reach + 2.0 ** -20
    if kw.get("softcap"):
        s_err += 2.0 ** -19 * reach.clamp(max=kw["softcap"])
    if q.dtype == BF16 and k.dtype == E4M3:
        most = torch.stack([R.gather(k, table[b], int(n)).abs().sum(-1).amax(-1) for b, n in enumerate(lens)])  # [B, Hkv]
        most = most.repeat_interleave(q.shape[1] // k.shape[1], 1) * abs(kw.get("q_scale", 1.0)) / q.shape[2] ** 0.5
        s_err += 2.0 ** -40 * q.double().abs().amax(-1) * most
    fin = torch.finfo(got.dtype)
    w = 2.0 ** -16 if v.dtype == BF16 else 2.0 ** -22
    tol = fin.eps / 2 * out.abs() + (1 + fin.eps) * (w + 2 * s_err)[..., None] * mag + fin.smallest_normal * fin.eps
    if v.dtype != BF16:  # an f16 term is nowhere finer than 2^-24, the largest weight 2^14
        tol += 2.0 ** -39 * R.visible_magnitude(v, table, lens, q.shape[1], **kw)
    err = (got.double() - out).abs()
    assert (err <= tol).all(), f"out: worst {float((err / tol).max()):.2f} of the bound"
    e, t = (lse.cpu().double() - want_lse).abs(), s_err + 2.0 ** -20 * want_lse.abs()
    assert (e <= t).all(), f"lse: worst {float((e / t).max()):.2f} of the bound"


def plain(lens, **kw):
    return make(lens, poison=False, **kw)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [4, 16])
@pytest.mark.parametrize("dtype,cache", [(BF16, E4M3), (F16, E4M3), (F16, F16), (BF16, BF16)])
def test_weights_keep_their_bits(dtype, cache, group, d):
    """Scores near 0 over values of both signs: an output far below the values shows what the weights lost."""
    check(plain([8, 5, 24, 300], hq=group, hkv=1, d=d, dtype=dtype, cache=cache, spread=0.02, seed=d + group))


@pytest.mark.parametrize("up", [10, 20, 28])
def test_bf16_query_elements_far_below_the_largest(up):
    """One element of a row 2^up times the others, where the keys are zero: the others make the scores."""
    q, k, v, table, lens = plain([80, 33], dtype=BF16, cache=E4M3, seed=up)
    q[..., 5] = 2.0 ** up
    k[..., 5] = 0
    check((q, k, v, table, lens), q_scale=1 / 16)


@pytest.mark.parametrize("softcap", [0.5, 50.0, 1e3, 1e6, 3e38])
@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, E4M3)])
@pytest.mark.parametrize("spread", [0.05, 4.0])
def test_caps_of_any_size(softcap, dtype, cache, spread):
    """A cap far above the scores leaves them as they are."""
    check(plain([300, 5], dtype=dtype, cache=cache, spread=spread, seed=3), softcap=softcap, q_scale=1 / 16 if cache == E4M3 else 1.0)
