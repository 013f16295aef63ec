"""What the roundings that include/qbd.h states leave of kv_attention's results on inputs that bring them out: against the
float64 reference, within the bound that follows from them."""
import numpy as np
import pytest
import torch

import block_quantized_decode_amd as qbd
from kv_util import DTYPES, Cache, check_attention, device, gpu, kv, note
from test_gpu_kv import FORMATS, layout

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kbits,vbits", FORMATS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 9, 40])
def test_fp32_scores_of_keys_with_an_outlier_that_the_query_compensates(new, dim, kbits, vbits):
    """Keys whose blocks hold one large channel and nothing beside it, queries with a mean that are small in that channel:
    the score is a sum of small terms, and the large ones of the query meet codes of zero."""
    rng = np.random.default_rng(dim + new)
    lens, page, heads, group = [5, 41, 60], 16, 2, 3
    table, pages = layout(rng, page, lens)
    cache = Cache(rng, pages, heads, page, dim, kbits, vbits)
    top, nb = kv.LEVELS[kbits], dim // 32
    at = np.arange(nb) * 32 + rng.integers(0, 32, size=nb)
    cache.codes[0][:] = 0
    cache.codes[0][..., at] = rng.choice([-top, top], size=(pages, heads, page, nb))
    cache.scales[0][:] = rng.uniform(0.2, 0.3, size=cache.scales[0].shape)
    cache.upload()
    q = (40 + 20 * rng.standard_normal((3 * new, heads * group, dim))).astype(np.float32)
    q[..., at] = rng.standard_normal((3 * new, heads * group, nb)) * 0.5 / top
    starts = (np.arange(4) * new).astype(np.int32)
    note("kv attention compensated outliers", new, dim, kbits, vbits)
    ref, mass, reach = kv.attention(q.astype(np.float64), cache.k, cache.v, table, lens, starts, scale=1.0)
    for hints in ({}, dict(max_q=new, max_len=60)):
        out = qbd.kv_attention(gpu(q), *cache.planes, gpu(table), gpu(np.array(lens, dtype=np.int32)), q_starts=gpu(starts), scale=1.0, **hints)
        check_attention("compensated outliers", out, ref, mass, reach, 60, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("vbits", [4, 8])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 9])
def test_16_bit_scores_of_keys_with_an_outlier_that_the_query_compensates(new, dim, vbits, dtype):
    """The same with rows of 16 bits, whose factors keep 11, and a mean further above the outlier's channel."""
    rng = np.random.default_rng(dim + new)
    lens, page, heads, group = [5, 41, 60], 16, 2, 3
    table, pages = layout(rng, page, lens)
    cache = Cache(rng, pages, heads, page, dim, 8, vbits)
    nb = dim // 32
    at = np.arange(nb) * 32 + rng.integers(0, 32, size=nb)
    cache.codes[0][:] = 0
    cache.codes[0][..., at] = rng.choice([-127, 127], size=(pages, heads, page, nb))
    cache.scales[0][:] = rng.uniform(0.2, 0.3, size=cache.scales[0].shape)
    cache.upload()
    q = 400 + 200 * rng.standard_normal((3 * new, heads * group, dim))
    q[..., at] = rng.standard_normal((3 * new, heads * group, nb)) * 0.5 / 127
    q = torch.from_numpy(q.astype(np.float32)).to(device()).to(DTYPES[dtype])
    starts = (np.arange(4) * new).astype(np.int32)
    note("kv attention compensated outliers", new, dim, vbits, dtype)
    ref, mass, reach = kv.attention(q.double().cpu().numpy(), cache.k, cache.v, table, lens, starts, scale=1.0)
    for hints in ({}, dict(max_q=new, max_len=60)):
        out = qbd.kv_attention(q, *cache.planes, gpu(table), gpu(np.array(lens, dtype=np.int32)), q_starts=gpu(starts), scale=1.0, **hints)
        check_attention("compensated outliers", out, ref, mass, reach, 60, dtype, np.abs(cache.v).max())


HEADS, GROUP = 8, 2


def prompt(cache, table, lens, news, q, window=0):
    """Rows enough for the prompt kernel, where news are."""
    starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    return qbd.kv_attention(q, *cache.planes, gpu(table), gpu(np.array(lens, dtype=np.int32)), q_starts=gpu(starts), max_q=max(news),
                            max_len=32768, window=window, scale=1.0), starts


def queries(rng, tokens, dim, dtype, spread):
    q = torch.from_numpy((rng.standard_normal((tokens, HEADS * GROUP, dim)) * spread).astype(np.float32)).to(device()).to(dtype)
    return q, q.double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("news", [[1, 1], [9, 5], [300, 280]])
@pytest.mark.parametrize("dim,kbits", [(64, 4), (128, 8), (256, 4)])
def test_small_elements_of_a_query_keep_their_bits(dim, kbits, news, dtype):
    """A channel whose queries are a millionth of their row's others, and whose keys are as much larger."""
    rng = np.random.default_rng(dim + 2)
    lens, page = [330, 290], 32
    table, pages = layout(rng, page, lens)
    cache = Cache(rng, pages, HEADS, page, dim, kbits, 4, kscale=(1e-5, 3e-5))
    codes, scales = cache.codes[0].reshape(pages, HEADS, page, dim // 32, 32), cache.scales[0]
    large = rng.random(scales.shape) < 0.1
    codes[large] = 0
    codes[large, 5], codes[large, 21] = 1, -1
    scales[large] = rng.uniform(100, 250, size=int(large.sum()))
    cache.upload()
    q, _ = queries(rng, sum(news), dim, DTYPES[dtype], 3000.0)
    q.view(*q.shape[:2], -1, 32)[..., [5, 21]] *= 1e-6
    note("kv small elements of a query", dim, kbits, news, dtype)
    out, starts = prompt(cache, table, lens, news, q)
    ref, mass, reach = kv.attention(q.double().cpu().numpy(), cache.k, cache.v, table, lens, starts, scale=1.0)
    check_attention("small elements", out, ref, mass, reach, max(lens), dtype, np.abs(cache.v).max())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,kbits,vbits", [(64, 4, 4), (96, 8, 4), (128, 4, 4), (128, 8, 8), (192, 8, 4), (256, 8, 8)])
def test_prompts_keep_small_values_beside_large_scales(dim, kbits, vbits, dtype):
    """V blocks with a scale above 256 here and there, some with small codes in them, among values of a thousandth."""
    rng = np.random.default_rng(dim)
    lens, news, page = [330, 290], [300, 280], 32
    table, pages = layout(rng, page, lens)
    cache = Cache(rng, pages, HEADS, page, dim, kbits, vbits, kscale=(0.002, 0.01), vscale=(2e-4, 2e-3))
    codes, scales = cache.codes[1].reshape(pages, HEADS, page, dim // 32, 32), cache.scales[1]
    large = rng.random(scales.shape) < 0.03
    scales[large] = rng.uniform(300, 60000, size=int(large.sum()))
    codes[large] = 0
    cache.upload()
    q, q64 = queries(rng, sum(news), dim, DTYPES[dtype], 1.0)
    note("kv prompts small beside large", dim, kbits, vbits, dtype)
    out, starts = prompt(cache, table, lens, news, q)
    ref, mass, reach = kv.attention(q64, cache.k, cache.v, table, lens, starts, scale=1.0)
    check_attention("V", out, ref, mass, reach, max(lens), dtype, np.abs(cache.v).max())
    # and the large blocks themselves, where the output's type holds them
    codes[large] = np.where(rng.random(codes[large].shape) < 0.1, 1, 0)
    scales[large] = rng.uniform(300, 1000, size=int(large.sum()))
    cache.upload()
    out, starts = prompt(cache, table, lens, news, q)
    ref, mass, reach = kv.attention(q64, cache.k, cache.v, table, lens, starts, scale=1.0)
    check_attention("large V", out, ref, mass, reach, max(lens), dtype, np.abs(cache.v).max())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,kbits,vbits", [(64, 4, 4), (96, 8, 4), (128, 4, 4), (128, 8, 8), (192, 8, 4), (256, 8, 8)])
def test_prompts_keep_small_keys_beside_large_scales(dim, kbits, vbits, dtype):
    """K blocks with a scale above 256 here and there, of zeros or of one small code, among scales of 1e-5 that queries in
    the thousands make up for."""
    rng = np.random.default_rng(dim + 1)
    lens, news, page = [330, 290], [300, 280], 32
    table, pages = layout(rng, page, lens)
    cache = Cache(rng, pages, HEADS, page, dim, kbits, vbits, kscale=(1e-5, 3e-5))
    codes, scales = cache.codes[0].reshape(pages, HEADS, page, dim // 32, 32), cache.scales[0]
    large = rng.random(scales.shape) < 0.03
    scales[large] = rng.uniform(300, 60000, size=int(large.sum()))
    codes[large] = 0
    cache.upload()
    q, q64 = queries(rng, sum(news), dim, DTYPES[dtype], 3000.0)
    note("kv prompts small keys beside large", dim, kbits, vbits, dtype)
    out, starts = prompt(cache, table, lens, news, q)
    ref, mass, reach = kv.attention(q64, cache.k, cache.v, table, lens, starts, scale=1.0)
    check_attention("K", out, ref, mass, reach, max(lens), dtype, np.abs(cache.v).max())
    # the large blocks take part: one code, in a channel whose queries are small
    codes[large, 5] = 1
    scales[large] = rng.uniform(300, 1000, size=int(large.sum()))
    q.view(*q.shape[:2], -1, 32)[..., 5] *= 1e-6
    cache.upload()
    out, starts = prompt(cache, table, lens, news, q)
    ref, mass, reach = kv.attention(q.double().cpu().numpy(), cache.k, cache.v, table, lens, starts, scale=1.0)
    check_attention("large K", out, ref, mass, reach, max(lens), dtype, np.abs(cache.v).max())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("window", [0, 37])
@pytest.mark.parametrize("news", [[1, 1, 1], [9, 5, 7], [300, 280, 260]])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_hidden_bytes_change_no_bit(dim, news, window, dtype):
    """NaN, infinite, large and ordinary scales in every place that no row sees: past a sequence's end, before its first
    row's window, in pages that it does not hold and where page 0 stands for those; the visible scales are small."""
    rng = np.random.default_rng(dim + window)
    lens, page = [330, 301, 275], 32
    table, pages = layout(rng, page, lens)
    pages += 1
    table = np.where(table >= 0, table + 1, table)  # page 0 is nobody's
    table[0, [2, 10]], table[1, 8] = -1, pages + 5
    cache = Cache(rng, pages, HEADS, page, dim, 8, 4, kscale=(1e-4, 1e-3), vscale=(1e-4, 1e-3))
    hidden = np.ones((pages, page), bool)
    for b, (n, new) in enumerate(zip(lens, news)):
        first = max(0, n - new + 1 - window) if window else 0
        for t in range(first, n):
            if 0 <= table[b, t // page] < pages:
                hidden[table[b, t // page], t % page] = False
    q, q64 = queries(rng, sum(news), dim, DTYPES[dtype], 30.0)
    note("kv hidden bytes", dim, news, window, dtype)
    clean, starts = prompt(cache, table, lens, news, q, window)
    ref, mass, reach = kv.attention(q64, cache.k, cache.v, table, lens, starts, window=window, scale=1.0)
    check_attention("clean", clean, ref, mass, reach, max(lens), dtype, np.abs(cache.v).max())
    for fill in ([300.0, 40000.0], [np.nan, np.inf, -np.inf], [0.5, 3.0, 1e-7], [np.nan, 500.0, 2e-4, 0.0]):
        for codes, scales in zip(cache.codes, cache.scales):
            at = np.broadcast_to(hidden[:, None], scales.shape[:3])
            scales[at] = rng.choice(fill, size=(int(at.sum()), scales.shape[3])).astype(np.float16)
            codes[at] = rng.integers(-7, 8, size=(int(at.sum()), dim))
        cache.upload()
        assert torch.equal(prompt(cache, table, lens, news, q, window)[0], clean), fill


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("news", [[1, 1], [9, 5], [300, 280]])
def test_queries_near_the_types_largest(news, dtype):
    """Scores of 10^37: the key with the largest takes all of its row, and nothing overflows."""
    rng = np.random.default_rng(7)
    lens, page, dim = [330, 290], 32, 64
    table, pages = layout(rng, page, lens)
    cache = Cache(rng, pages, HEADS, page, dim, 8, 8)
    q, q64 = queries(rng, sum(news), dim, DTYPES[dtype], 1e36)
    starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    note("kv large queries", news, dtype)
    out = qbd.kv_attention(q, *cache.planes, gpu(table), gpu(np.array(lens, dtype=np.int32)), q_starts=gpu(starts), max_q=max(news),
                           max_len=32768).double().cpu().numpy()
    ref, _, _ = kv.attention(q64, cache.k, cache.v, table, lens, starts)
    assert np.isfinite(out).all()
    # two keys whose scores are closer than the factors' 11 bits may change places: that is a few rows in a thousand; the
    # values' own roundings are the output's, and for prompts the 11 bits of V
    unit = {"f32": 2.0 ** -22, "bf16": 2.0 ** -8 + 2.0 ** -11}[dtype]
    other = (np.abs(out - ref) > unit * np.abs(ref) + 1e-30).any(-1)
    assert other.mean() < 0.02, other.mean()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vscale", [(0.02, 0.3), (1e-6, 4e-5), (1000.0, 8000.0)])
@pytest.mark.parametrize("news", [[1, 1], [300, 280]])
def test_large_scores_of_every_size(news, vscale, dtype):
    """Scores of 10^6 to 10^11, where a reference is rounded to units of less than one up to many thousands: finite, and the
    key with the largest takes all of its row."""
    rng = np.random.default_rng(8)
    lens, page, dim = [330, 290], 32, 64
    table, pages = layout(rng, page, lens)
    cache = Cache(rng, pages, HEADS, page, dim, 8, 8, vscale=vscale)
    starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    q0 = rng.standard_normal((sum(news), HEADS * GROUP, dim))
    for spread in (1e6, 5e6, 1e7, 3e7, 6e7, 1e8, 1.5e8, 2e8, 3e8, 4e8, 6e8, 1e9, 1e11):
        q = torch.from_numpy((q0 * spread).astype(np.float32)).to(device()).to(DTYPES[dtype])
        note("kv large scores", news, vscale, dtype, spread)
        out = qbd.kv_attention(q, *cache.planes, gpu(table), gpu(np.array(lens, dtype=np.int32)), q_starts=gpu(starts), max_q=max(news),
                               max_len=32768).double().cpu().numpy()
        ref, _, _ = kv.attention(q.double().cpu().numpy(), cache.k, cache.v, table, lens, starts)
        assert np.isfinite(out).all(), spread
        # as above: values by their own roundings, but for a few rows whose two largest scores are closer than the factors' bits;
        # 16-bit rows' weights times small V scales (below 2^-14 a binary16 product has a fixed step) by 2^-25 of 127
        unit = {"f32": 2.0 ** -22, "bf16": 2.0 ** -8 + 2.0 ** -11}[dtype]
        step = {"f32": 1e-30, "bf16": 127 * 2.0 ** -25}[dtype]
        other = (np.abs(out - ref) > unit * np.abs(ref) + step).any(-1)
        assert other.mean() < 0.02, (spread, other.mean())
