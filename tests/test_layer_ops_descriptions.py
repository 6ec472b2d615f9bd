"""Sizes that a 32-bit field of a description would cut off are refused."""

import pytest
import torch

import activation_sparse_tiered_amd as spax

BIG = 2 ** 32 + 3      # 3 once cut to 32 bits


def _rows(n, d, dtype=torch.float16):
    return torch.zeros((), dtype=dtype).expand(n, d)


def _attention(**kw):
    k = torch.zeros(8, 2, 16, 64, dtype=torch.float16)
    cache = spax.make_kv_cache(k, k.clone(), torch.zeros(3, 4, dtype=torch.int32))
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    return spax.make_attention(cache, q, torch.zeros(3, dtype=torch.int32), q.clone(), **kw)


def test_sizes_past_32_bits_are_refused_not_cut():
    x = _rows(BIG, 1)
    with pytest.raises(ValueError, match="n_rows"):
        spax.make_glu(x, x, x)
    with pytest.raises(ValueError, match="n_rows"):
        spax.make_residual_norm(x, x, x, x)
    with pytest.raises(ValueError, match="max_len"):
        _attention(max_len=BIG)
    with pytest.raises(ValueError, match="window"):
        _attention(window=BIG)
    row = torch.zeros(1, 1, 64, dtype=torch.float16).expand(BIG, 1, 64)
    k = torch.zeros(8, 1, 16, 64, dtype=torch.float16)
    table = torch.zeros(3, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="n_tokens"):
        spax.make_kv_append(spax.make_kv_cache(k, k.clone(), table), None, row, row,
                            torch.zeros(3, dtype=torch.int32), None)
    pages = k[:1].expand(BIG, 1, 16, 64)
    with pytest.raises(ValueError, match="n_pages"):
        spax.make_kv_cache(pages, pages, table)
    with pytest.raises(ValueError, match="n_seqs"):
        spax.make_kv_cache(k, k.clone(), table[:1].expand(BIG, 4))


def test_the_largest_sizes_of_the_fields_are_taken():
    assert spax.make_glu(*[_rows(2 ** 31 - 1, 1)] * 3).n_rows == 2 ** 31 - 1
    assert _attention(max_len=2 ** 31 - 1).max_len == 2 ** 31 - 1
