"""Windowed attention with queries far from unit size: the scores are those of Q and `scale`
together, so a query 2^k times as large with a scale 2^-k as large is the same call."""
import numpy as np
import pytest
import torch

import rotated_bit_kv_isoquant_b200 as iq
from _window_ref import dequantize_pages, window_attention
from test_gpu_window import DT, Case

pytestmark = pytest.mark.gpu

# the kernels behind them: one query token, row blocks, tensor memory with one and two row blocks
FORMS = [dict(n_q=1), dict(n_q=3), dict(n_q=20), dict(n_q=40), dict(n_q=1, bits=4), dict(n_q=3, bits=4),
         dict(n_q=20, bits=2), dict(n_q=1, bits=2), dict(n_q=40, bits=4), dict(n_q=1, d=256), dict(n_q=5, d=256)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def run(c, Q, scale):
    out = torch.full(Q.shape, float("nan"), dtype=DT[c.out_t], device="cuda")
    iq.isoq_multi_token_attention_window(c.params, c.cache, Q, c.sl, c.max_len, c.W, c.S, out, scale, c.workspace())
    return out


def check(c, oracle, Q, scale, got):
    p64 = oracle.make_params_v(c.seed, c.d, c.hkv, c.rot)[1].astype(np.float64)
    pages = dequantize_pages(oracle, p64, c.blocks, c.d, c.bits, c.rot)
    ref, tol = window_attention(pages, c.pt.numpy(), c.lens, Q.float().cpu().numpy().astype(np.float64), scale,
                                c.W, c.S, c.bits, c.out_t)
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    err = np.linalg.norm(got - ref, axis=-1)
    assert (err <= tol).all(), f"worst {np.max(err / tol)}, {np.argwhere(err > tol)[:4]}"
    assert iq.isoq_get_status(c.cache) == 0


@pytest.mark.parametrize("k", [-80, -60, -30, -14, -8, 8, 11, 14, 30, 60, 94])
@pytest.mark.parametrize("i", range(len(FORMS)))
def test_a_query_and_its_scale_by_powers_of_two(oracle, i, k):
    c = Case([300, 190], 12, 3, 150, 4, q="bf16" if i % 2 else "f32", out="f32", seed=i, **FORMS[i])
    Q, scale = c.Q * 2.0 ** k, c.d ** -0.5 * 2.0 ** -k
    check(c, oracle, Q, scale, run(c, Q, scale))


@pytest.mark.parametrize("i", range(len(FORMS)))
def test_rows_of_very_different_sizes(oracle, i):
    """Query rows of a call from 2^-30 to 2^30, each against its own bound: one row's size takes
    nothing from another's."""
    c = Case([300, 190], 12, 3, 150, 4, q="f32", out="f32", seed=20 + i, **FORMS[i])
    k = torch.randint(-30, 31, c.Q.shape[:-1], generator=torch.Generator().manual_seed(i)).cuda()
    Q = c.Q * torch.exp2(k.float())[..., None]
    check(c, oracle, Q, c.d ** -0.5, run(c, Q, c.d ** -0.5))


@pytest.mark.parametrize("i", range(len(FORMS)))
def test_zero_queries_and_fp16_ones_near_their_largest(oracle, i):
    c = Case([300, 190], 12, 3, 150, 4, q="f16", out="f32", seed=40 + i, **FORMS[i])
    Q = c.Q.sign() * 60000.0          # the largest rotated element: up to sqrt(d) times as large
    Q[:, :, ::3] = 0
    scale = c.d ** -0.5 * 2.0 ** -16
    check(c, oracle, Q, scale, run(c, Q, scale))


@pytest.mark.parametrize("k", [-30, 14])
@pytest.mark.parametrize("f", [dict(n_q=3), dict(n_q=12), dict(n_q=50), dict(n_q=1, bits=4), dict(n_q=3, bits=2)])
def test_queries_with_the_window_in_several_chunks(oracle, f, k):
    c = Case([9000], 8, 2, 8000, 4, q="f32", out="f32", seed=70, **f)
    Q, scale = c.Q * 2.0 ** k, c.d ** -0.5 * 2.0 ** -k
    check(c, oracle, Q, scale, run(c, Q, scale))


def test_a_row_that_is_not_finite_stays_alone():
    """NaN and infinite queries give rows that are not finite; every other row keeps its bits."""
    for n_q, bits in ((1, 3), (3, 3), (40, 3), (100, 3), (3, 4), (40, 4)):
        c = Case([300, 190], 8, 2, 150, 4, n_q=n_q, bits=bits, q="f32", out="f32", seed=80, poison=False)
        want = run(c, c.Q, c.d ** -0.5)
        Q = c.Q.clone()
        Q[0, n_q // 2, 3, 5], Q[1, 0, 7, 100] = float("nan"), float("inf")
        got = run(c, Q, c.d ** -0.5)
        bad = torch.zeros(Q.shape[:-1], dtype=torch.bool)
        bad[0, n_q // 2, 3] = bad[1, 0, 7] = True
        assert torch.equal(got[~bad.cuda()], want[~bad.cuda()]), (n_q, bits)
