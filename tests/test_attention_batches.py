"""Attention over the key-value cache for batches of more sequences than a CTA
has threads (the plan then takes them in blocks), with runs of sequences that
have no rows, and batches that mix single tokens with chunks: each kernel,
against the definition in 64 bits."""
import ctypes
import random

import pytest
import torch

import int4_weight_mixed_gb300 as w4
import kv
from fake_cuda import build
from test_attention import _attend, _check, _tree
from test_kv_cache import _cache, _of

S8, F8 = torch.int8, torch.float8_e4m3fn
DEC, UNPACKED, OWN = "attn_dec_kernel", "attn_unpack_kernel", "attn_tc_kernel"


def _ragged(B, most, longest, seed):
    """Rows and lengths of B sequences: runs of sequences without rows (at the
    start, the end and across multiples of 128), then up to `most` rows each."""
    r = random.Random(seed)
    rows, lens = [], []
    while len(rows) < B:
        run = r.randint(1, 40)
        none = r.random() < 0.4 or not rows
        for _ in range(run):
            n = 0 if none else r.randint(1, most)
            rows.append(n)
            lens.append(r.randint(max(n, 1), longest) if n or r.random() < 0.5 else 0)
    rows, lens = rows[:B], lens[:B]
    for b in range(126, min(B, 131)):  # ... and around the first block's end
        rows[b], lens[b] = (0, 7) if b % 2 else (1, 300)
    if not any(rows):
        rows[0] = lens[0] = 1
    return rows, lens


# sequences, most rows, longest, query heads, key heads, dimension, table width
# (0: as wide as the longest sequence), kernel
CASES = [
    (127, 1, 500, 8, 2, 128, 0, DEC), (128, 1, 500, 8, 2, 128, 0, DEC),
    (129, 1, 500, 8, 2, 128, 0, DEC), (129, 1, 400, 6, 2, 64, 0, DEC),
    (300, 1, 300, 4, 1, 64, 0, DEC), (700, 1, 200, 4, 1, 128, 0, DEC),
    (700, 2, 200, 16, 2, 64, 0, DEC),
    (321, 9, 200, 16, 1, 64, 4096, OWN), (330, 9, 300, 16, 1, 128, 1024, OWN),
    (645, 9, 150, 16, 1, 128, 1024, OWN), (700, 9, 150, 8, 1, 64, 4096, OWN),
    (330, 260, 280, 12, 1, 128, 0, UNPACKED), (330, 260, 280, 12, 1, 64, 0, UNPACKED),
]


def _batch(B, most, longest, width, page=32, behind=2):
    rows, lens = _ragged(B, most, longest, 7 * B + most)
    batch = kv.Batch(rows, lens, page, seed=B, behind=behind)
    if width > batch.width:
        batch.table = torch.nn.functional.pad(batch.table, (0, width - batch.width), value=-1)
        batch.width = width
    return batch


def _kernels(rec, heads, kv_heads, dim, rows, sequences, width, page=32, **kw):
    rec.reset()
    cache = _cache(heads=kv_heads, head_dim=dim, page_size=page)
    st = rec.lib.w4_cache_attention(
        ctypes.byref(cache), ctypes.byref(_of(table_width=width, sequences=sequences)),
        0x80000000, w4.F16, rows, heads, heads * dim, 0.1, 0, 0, 1 << 40, 1 << 41,
        kw.get("nws", 1 << 32), None)
    assert st == w4.OK, rec.lib.w4_last_error()
    return " ".join(k for _, k in rec.launches())


@pytest.fixture(scope="module")
def rec(tmp_path_factory):
    return build(tmp_path_factory.mktemp("recorded"))


@pytest.mark.parametrize("case", CASES)
def test_kernel_of_the_case(rec, case):
    """The cases below run on the kernels that they are meant for."""
    B, most, longest, Hq, Hkv, D, width, kernel = case
    batch = _batch(B, most, longest, width)
    got = _kernels(rec, Hq, Hkv, D, batch.T, B, batch.width)
    assert kernel in got
    assert (UNPACKED in got) == (kernel == UNPACKED) and (DEC in got) == (kernel == DEC)


@pytest.mark.gpu
@pytest.mark.parametrize("codes,dt", [(S8, torch.bfloat16), (F8, torch.float16)])
@pytest.mark.parametrize("case", CASES)
def test_many_sequences(gpu_lib, case, codes, dt):
    B, most, longest, Hq, Hkv, D, width, _ = case
    batch = _batch(B, most, longest, width)
    _check(batch.rows, batch.lens, Hq, Hkv, D, 32, codes, dt, batch=batch)


@pytest.mark.gpu
@pytest.mark.parametrize("D,width", [(128, 0), (64, 0), (128, 1024), (64, 4096)])
def test_many_trees(gpu_lib, D, width):
    batch = _batch(330, 9, 200, width)
    _check(batch.rows, batch.lens, 16, 1, D, 32, S8, torch.bfloat16, 50, 3,
           _tree(batch.rows, 9), batch=batch)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("codes,dt", [(S8, torch.bfloat16), (F8, torch.float16)])
def test_tokens_beside_chunks(gpu_lib, D, codes, dt, wide):
    """Single tokens of many sequences and a few chunks, of every position among
    them, in one call."""
    r = random.Random(D)
    rows = [1] * 90
    for b, n in ((0, 300), (40, 65), (41, 129), (89, 520)):
        rows[b] = n
    lens = [max(n, r.randint(1, 900)) for n in rows]
    _check(rows, lens, 8, 2, D, 64, codes, dt, wide=wide)
    _check(rows, lens, 8, 2, D, 64, codes, dt, 100, 4, wide=wide)
