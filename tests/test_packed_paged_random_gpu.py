"""Packed and paged attention against 64 bits over random batches: lengths,
head layouts, types, masks, scales, pages and prefixes drawn together."""
import math
import random

import pytest

import exact_tiled_attention_04_gb300 as fa

from .gpu_util import ensure_library

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from . import test_packed_gpu as packed, test_paged_gpu as paged  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_library()


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert fa.fa_device_status(None) == fa.FA_OK


def log_uniform(r, lo, hi):
    return int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))


def heads(r):
    H_kv = r.choice([1, 2, 3, 5])
    return H_kv * r.choice([1, 2, 3, 4, 5, 7, 8]), H_kv, r.choice([64, 128]), r.choice(["bf16", "f16"])


def lengths(r, B, longest):
    return [0 if r.random() < 0.1 else log_uniform(r, 1, max(1, longest)) for _ in range(B)]


@pytest.mark.parametrize("seed", range(16))
def test_packed(seed):
    r = random.Random(seed)
    H, H_kv, d, dtype = heads(r)
    B = log_uniform(r, 1, 100)
    lens = lengths(r, B, 2 * log_uniform(r, B, 1200) // B)
    keys = [max(0, n + r.choice([0, 0, 1, -1, 130, -200, 500])) for n in lens] if r.random() < 0.5 else None
    batch = packed.batch(seed, lens, H, H_kv, d, dtype, keys)
    packed.check_backward(*batch, r.random() < 0.6, scale=r.choice([None, None, 0.0, -0.2, 0.7]))


@pytest.mark.parametrize("seed", range(16))
def test_steps(seed):
    r = random.Random(100 + seed)
    H, H_kv, d, dtype = heads(r)
    N_q = r.choice([1, 1, 1, 2, 3, 4, 8, 16])
    while N_q * H // H_kv > 128:
        N_q //= 2
    B = log_uniform(r, 1, 300)
    lens = lengths(r, B, 12000 // B)
    prefix = log_uniform(r, 1, 3000) if r.random() < 0.4 else 0
    g = paged.rng(seed)
    cache, pages = paged.cache_of(g, lens, H_kv, d, r.choice([16, 32, 64, 128]), dtype, prefix=prefix)
    paged.check(g, cache, lens, H, N_q, causal=N_q > 1 and r.random() < 0.6, prefix_pages=pages, prefix=prefix,
                scale=r.choice([None, None, -0.3, 0.0]))


@pytest.mark.parametrize("seed", range(12))
def test_rows_stored(seed):
    r = random.Random(200 + seed)
    H, H_kv, d, dtype = heads(r)
    B = log_uniform(r, 1, 40)
    held, new = lengths(r, B, 500), lengths(r, B, 200)
    new[0] = max(new[0], 1)
    rot = r.choice([d, d // 2, 16, 0])
    cache, _ = paged.cache_of(paged.rng(seed), held, H_kv, d, r.choice([16, 32, 64, 128]), dtype, room=max(new), poison=False)
    paged.check_append(paged.rng(seed), cache, new, r.choice([0, H]), fa.rotary_table(800, rot) if rot else None,
                       interleaved=r.random() < 0.5, with_k=r.random() < 0.5, in_place=r.random() < 0.5)
