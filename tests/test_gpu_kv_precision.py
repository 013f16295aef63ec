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
