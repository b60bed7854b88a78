"""Sizes that the windowed calls refuse have no workspace size, and the binding's numbers keep
their value on the way into the C interface's ints."""
import pytest
import torch

import rotated_bit_kv_isoquant_b200 as iq
from test_window_cpu import _Cache

f = iq.raw_lib().isoq_window_workspace_bytes


@pytest.mark.parametrize("hq,hkv,fits", [(64, 8, 4095), (16, 16, 4 * 4095), (8, 2, 32767), (32, 2, 2 * 4095)])
def test_rows_at_d256_are_counted_in_blocks_of_four(hq, hkv, fits):
    """d = 256 works on blocks of 4 rows: at most 65535 of them over the KV heads."""
    assert hkv * -(-fits * (hq // hkv) // 4) <= 65535 < hkv * -(-(fits + 4) * (hq // hkv) // 4)
    assert f(1, fits, hq, hkv, 256, 1000, 100, 4) > 0
    assert f(1, fits + 4, hq, hkv, 256, 1000, 100, 4) == 0
    assert f(1, fits + 4, hq, hkv, 128, 1000, 100, 4) > 0      # blocks of 8 and more


def test_more_sequences_than_a_grid_holds():
    assert f(65535, 1, 8, 2, 128, 1000, 100, 4) > 0
    assert f(65536, 1, 8, 2, 128, 1000, 100, 4) == 0


@pytest.mark.parametrize("n_q", [1, 3, 40])
def test_more_than_16_query_heads_a_kv_head(n_q):
    assert f(1, n_q, 32, 2, 128, 1000, 100, 4) > 0
    assert f(1, n_q, 34, 2, 128, 1000, 100, 4) == 0


@pytest.mark.parametrize("n_seqs,hq,hkv,d,W", [(1, 32, 4, 128, 1024), (8, 64, 8, 128, 4096), (32, 16, 8, 256, 900),
                                               (64, 32, 8, 128, 8192)])
def test_a_decode_that_merges_in_a_cluster_asks_for_no_partial_rows(n_seqs, hq, hkv, d, W):
    """One row of state per query row is asked for, as of a call with a single chunk; the chunks
    of these windows meet in shared memory."""
    assert f(n_seqs, 1, hq, hkv, d, 32768, W, 4) == n_seqs * hq * (d + 4) * 4


def test_numbers_beyond_an_int_are_not_wrapped():
    good = [1, 1, 8, 2, 128, 1000, 100, 4]
    assert iq.isoq_window_workspace_bytes(*good) > 0
    for i in range(len(good)):
        for n in (2 ** 31, 2 ** 32 + good[i], -2 ** 32 + good[i]):
            assert iq.isoq_window_workspace_bytes(*good[:i], n, *good[i + 1:]) == 0, (i, n)
    Q, lens, ws = torch.zeros(2, 8, 128), torch.zeros(2, dtype=torch.int32), torch.zeros(16)
    for n in (2 ** 31, 2 ** 32 + 16, -1):
        with pytest.raises(ValueError, match="max_seq_len"):
            iq.isoq_decode_attention_window(None, _Cache, Q, lens, n, 16, 4, Q, 1.0, ws)
        with pytest.raises(ValueError, match="max_seq_len"):
            iq.isoq_multi_token_attention_window(None, _Cache, Q[:, None], lens, n, 16, 4, Q[:, None], 1.0, ws)
