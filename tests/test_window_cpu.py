"""Host-side checks of the windowed attention: the reference that the GPU tests use against
the oracle, the workspace arithmetic, and what the calls refuse before any CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

import rotated_bit_kv_isoquant_b200 as iq
from _window_ref import dequantize_pages, visible, window_attention

LIB = iq.raw_lib()


def _random_pages(oracle, d, H, n_pages, bits, rot, seed):
    rng = np.random.default_rng(seed)
    _, p32 = oracle.make_params_v(seed, d, H, rot)
    p64 = p32.astype(np.float64)
    blocks = np.zeros((n_pages, H, oracle.block_bytes(d, bits=bits)), np.uint8)
    pt = rng.permutation(n_pages).astype(np.int32)[None]
    T = n_pages * 64
    K, V = rng.standard_normal((2, T, H, d)) * 3
    oracle.quantize_append(p64, d, H, 64, blocks, pt, K, V, np.zeros(T, np.int32),
                           np.arange(T, dtype=np.int32), bits=bits, rot=rot)
    return p64, blocks, pt


@pytest.mark.parametrize("d,bits,rot", [(128, 3, 0), (256, 3, 1), (128, 2, 1), (128, 4, 0)])
def test_reference_with_an_open_window_is_the_oracle_decode(oracle, d, bits, rot):
    p64, blocks, pt = _random_pages(oracle, d, 2, 3, bits, rot, 5)
    Q = np.random.default_rng(1).standard_normal((1, 1, 4, d))
    L = 150
    pages = dequantize_pages(oracle, p64, blocks, d, bits, rot)
    ref, tol = window_attention(pages, pt, [L], Q, d ** -0.5, 10 ** 9, 0, bits)
    want = oracle.decode_attention(p64, d, 2, 64, blocks, pt, [L], Q[:, 0], d ** -0.5, bits=bits, rot=rot)
    assert np.abs(ref[:, 0] - want).max() <= 1e-11 * np.abs(want).max()
    assert (tol < 2e-2 * np.linalg.norm(ref, axis=-1)).all() and (tol > 0).all()


def test_visible_tokens():
    assert visible(9, 3, 2).tolist() == [0, 1, 7, 8, 9]
    assert visible(9, 100, 2).tolist() == list(range(10))
    assert visible(3, 3, 2).tolist() == [0, 1, 2, 3]      # sinks and window overlap
    assert visible(0, 1, 4).tolist() == [0] and visible(-1, 5, 4).tolist() == []
    assert visible(9, 1, 0).tolist() == [9]


@pytest.mark.parametrize("n_q", [1, 5, 40, 300])
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (64, 8, 128), (16, 8, 256), (7, 7, 128)])
def test_workspace_grows_with_the_window_not_the_context(n_q, hq, hkv, d):
    def f(L, W, S):
        return iq.isoq_window_workspace_bytes(2, n_q, hq, hkv, d, L, W, S)
    unit = 2 * n_q * hq * (d + 4) * 4
    for L, W, S in [(0, 1, 0), (1, 1, 0), (100, 64, 4), (131072, 4096, 4), (131072, 2 ** 31 - 1, 0),
                    (2 ** 31 - 1, 1000, 2 ** 31 - 1)]:
        assert f(L, W, S) % unit == 0 and f(L, W, S) >= unit
    assert f(131072, 1024, 4) <= f(131072, 131072, 0)
    # a context shorter than the window needs no more than its own pages' chunks
    assert f(500, 4096, 64) <= unit * 8


def test_workspace_refuses():
    f = LIB.isoq_window_workspace_bytes
    assert f(1, 1, 8, 2, 128, 1000, 100, 4) > 0
    for bad in [(-1, 1, 8, 2, 128, 1000, 100, 4), (1, 0, 8, 2, 128, 1000, 100, 4),
                (1, 1, 7, 2, 128, 1000, 100, 4), (1, 1, 8, 0, 128, 1000, 100, 4),
                (1, 1, 8, 2, 96, 1000, 100, 4), (1, 1, 8, 2, 128, -1, 100, 4),
                (1, 1, 8, 2, 128, 1000, 0, 4), (1, 1, 8, 2, 128, 1000, 100, -1),
                (1, 2 ** 31 - 1, 8, 2, 128, 1000, 100, 4)]:
        assert f(*bad) == 0, bad


def test_window_calls_refuse_before_any_cuda_call():
    c = iq.isoq_cache(128, 2, 64, 4, 2, 1, None, None, None)
    assert LIB.isoq_decode_attention_window(None, ctypes.byref(c), None, 0, 1, 8, None, 64, 16, 0,
                                            None, 0, 1.0, None, 0, None) == iq.ISOQ_E_ARG
    assert LIB.isoq_multi_token_attention_window(None, ctypes.byref(c), None, 0, 1, 2, 8, None, 64,
                                                 16, 0, None, 0, 1.0, None, 0, None) == iq.ISOQ_E_ARG


class _Cache:
    d = 128
    blocks = torch.zeros(1)


def test_binding_checks_shapes_and_devices():
    Q, lens, ws = torch.zeros(2, 8, 128), torch.zeros(2, dtype=torch.int32), torch.zeros(16)
    call = iq.isoq_decode_attention_window
    for q, sl, out in [(Q[0], lens, Q[0]), (Q, lens, Q[:1]), (Q, lens[:1], Q),
                       (Q[..., :64], lens, Q[..., :64]), (Q, lens.to("meta"), Q)]:
        with pytest.raises(ValueError):
            call(None, _Cache, q, sl, 100, 16, 4, out, 1.0, ws)
    for W, S in [(0, 4), (2 ** 31, 4), (2 ** 32 + 16, 4), (16, -1), (16, 2 ** 31)]:
        with pytest.raises(ValueError):
            call(None, _Cache, Q, lens, 100, W, S, Q, 1.0, ws)
    with pytest.raises(ValueError):
        iq.isoq_multi_token_attention_window(None, _Cache, Q, lens, 100, 16, 4, Q, 1.0, ws)


def test_read_back_binding_checks():
    class C:
        d, n_kv_heads, blocks = 128, 2, torch.zeros(1)
    i = torch.zeros(3, dtype=torch.int32)
    K = torch.zeros(3, 2, 128)
    for sid, pos, k, v in [(i, i, None, None), (i, i[:2], K, K), (i[None], i[None], K, K), (i, i, K[:2], K),
                           (i, i, K, K.half()), (i, i, K[:, :1], None), (i, i, K.to("meta"), None)]:
        with pytest.raises(ValueError):
            iq.isoq_dequantize(None, C, sid, pos, k, v)
    with pytest.raises(ValueError):
        iq.isoq_dequantize_rope(None, C, i, i, K, K, torch.zeros(9, 32, 2))
    assert LIB.isoq_dequantize(None, None, None, None, 1, None, None, 0, None) == iq.ISOQ_E_ARG
