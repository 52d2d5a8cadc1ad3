"""GPU: gqa_paged_tree_attn over sequences so long that one block sums up thousands of tiles, against the plain 64-bit
form.  A few physical pages stand in the block tables many times, so that a million tokens need little memory and the
64-bit form counts each of them as often as it is seen."""
import math

import pytest
import torch

import gqa_attention_kv_split_gb300 as gqa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn
PAGE = 256


@pytest.fixture(scope="module", autouse=True)
def built():
    gqa.build()
    yield
    assert gqa.gqa_check_device_errors(0) == 0


def make(lens, n, hq, hkv, d, dtype, cache, rising, seed):
    """Drafts of n tokens in chains; elements of V are positive in its first half and of both signs in the other one."""
    g = torch.Generator().manual_seed(seed)
    num = 16
    q = torch.randn(n * len(lens), hq, d, generator=g).to(dtype)
    k, v = torch.randn(num, hkv, PAGE, d, generator=g), torch.randn(num, hkv, PAGE, d, generator=g)
    v[..., :d // 2] = v[..., :d // 2].abs() * 0.25 + 0.5
    if rising:  # (a page's first element of K rises with its number, and rows' maxima with it)
        k[..., 0] = torch.arange(num).view(-1, 1, 1) * 6.0
    if cache == E4M3:
        v *= 16
    k, v = k.to(cache), v.to(cache)
    cols = (max(lens) + PAGE - 1) // PAGE
    table = torch.randint(0, num, (len(lens), cols), generator=g)
    if rising:
        table = table.sort(1).values
    return q, k, v, table.to(torch.int32)


def plain(q, k, v, table, lens, n, rows):
    """out, lse and sum p |v| of the given rows, float64; f: how often a row sees each place of the pages."""
    T, hq, d = q.shape
    hkv = k.shape[1]
    ks, vs = (x.double().permute(1, 0, 2, 3).reshape(hkv, -1, d).repeat_interleave(hq // hkv, 0) for x in (k, v))
    out, lse, mag, reach = [], [], [], []
    for t in rows:
        b, end = t // n, lens[t // n] - n + t % n + 1
        f = torch.zeros(k.shape[0], PAGE, dtype=torch.float64)
        f += torch.bincount(table[b, :end // PAGE].long(), minlength=k.shape[0])[:, None]
        if end % PAGE:
            f[table[b, end // PAGE].long(), :end % PAGE] += 1
        s = torch.einsum("hd,hnd->hn", q[t].double(), ks) / math.sqrt(d) + f.view(-1).log()
        lse.append(torch.logsumexp(s, -1))
        p = torch.exp(s - lse[-1][:, None])
        out.append(torch.einsum("hn,hnd->hd", p, vs))
        mag.append(torch.einsum("hn,hnd->hd", p, vs.abs()))
        reach.append(torch.einsum("hd,hnd->hn", q[t].double().abs(), ks.abs()).amax(-1) / math.sqrt(d))
    return (torch.stack(x) for x in (out, lse, mag, reach))


def check(lens, n, hq, hkv, d, dtype, cache, rising=False, seed=0):
    """The bound: half a step of the output; a weight's two terms (2^-16 in bf16) and the scores' error as in
    paged_reference; the product with V, whose accumulator takes two sums for 16 tokens, each off by 2^-23 of what has
    been summed, for 16384 tokens at most before it is added to a sum in f32, one rounding (2^-24) for 16384 tokens; and
    the sum of the weights: 64 additions (2^-24) within a tile of 128 tokens (64 at head dim 256), and one for every other
    tile."""
    q, k, v, table = make(lens, n, hq, hkv, d, dtype, cache, rising, seed)
    T = q.shape[0]
    lse = torch.full((T, hq), 9.0, device=DEV)
    got = gqa.gqa_paged_tree_attn(q.to(DEV), k.to(DEV), v.to(DEV), table.to(DEV), torch.arange(0, T + 1, n, dtype=torch.int32, device=DEV),
                                  torch.tensor(lens, dtype=torch.int32, device=DEV), lse=lse)
    torch.cuda.synchronize()
    rows = sorted({0, T - 1, n * (len(lens) // 2) + n // 2})
    out, want_lse, mag, reach = plain(q, k, v, table, lens, n, rows)
    assert torch.isfinite(got).all()
    eps = torch.finfo(dtype).eps
    s_err = 2.0 ** -19 * reach + 2.0 ** -20
    sums = 2.0 ** -23 * min(max(lens), 16384) / 8 + 2.0 ** -24 * max(lens) / 16384
    weights = 2.0 ** -24 * (max(lens) / (128 if d == 256 else 256) + 64)
    tol = eps / 2 * out.abs() + (1 + eps) * (2.0 ** -16 + sums + weights + 2 * s_err)[..., None] * mag
    err = (got.cpu()[rows].double() - out).abs()
    assert (err <= tol).all(), f"out: worst {float((err / tol).max()):.2f} of the bound, {float((err / mag).max()):.2e} of sum p |v|"
    e = (lse.cpu()[rows].double() - want_lse).abs()
    assert (e <= s_err + weights + 2.0 ** -20 * want_lse.abs()).all()
    # What a long sum is off by does not go to one side: the mean over the elements of one sign is far below a step.
    rel = ((got.cpu()[rows].double() - out) / out)[..., :d // 2]
    drift = abs(float(rel.mean()))
    assert drift <= eps / 2 / math.sqrt(rel.numel()) * 4 + float(sums + weights + 2.0 ** -16) / 2, drift
    return got


LONG = 1 << 20


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3)])
def test_a_million_tokens_in_one_sum(dtype, cache, d):
    """More sequences than gangs of blocks: each unit is one block's, from its first tile to its last."""
    lens = [LONG] * 19
    check(lens, 4, 32, 8, d, dtype, cache, seed=d)


@pytest.mark.parametrize("n,hq", [(1, 8), (8, 64), (16, 64), (40, 32)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_in_copies_and_in_blocks(n, hq, d):
    """8, 64 and 128 rows a KV head, in four copies, two (or none), one, and 160 in two blocks."""
    check([300000 - 1000 * i for i in range(19)], n, hq, 8, d, F16, F16, seed=n)


@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, E4M3)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_maxima_that_rise_between_the_sums(dtype, cache, d):
    check([200000] * 19, 4, 32, 8, d, dtype, cache, rising=True, seed=d)


@pytest.mark.parametrize("tokens", [16384, 16385, 16512, 32768, 32769, 49153])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_around_the_sums_own_lengths(tokens, d):
    check([tokens] * 20, 3, 16, 8, d, F16, F16, seed=d)


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_pieces_with_several_sums(cache, hkv):
    """Long sequences in several blocks' shares, whose first and last pieces both go through sums of their own."""
    check([500000, 9000, 700001, 400000, 123], 6, 4 * hkv, hkv, 128, BF16, cache, seed=hkv)
    check([900000], 20, 4 * hkv, hkv, 64, BF16, cache, rising=True, seed=hkv)


def test_same_bits_every_time():
    want = check([400000, 300000, 200000], 5, 32, 8, 128, F16, F16, seed=3)
    for _ in range(3):
        assert torch.equal(check([400000, 300000, 200000], 5, 32, 8, 128, F16, F16, seed=3), want)
