"""The windowed calls at the ends of what they accept: sizes at the grid's limits, a workspace of
exactly the size asked for, and lengths next to the largest position."""
import numpy as np
import pytest
import torch

import rotated_bit_kv_isoquant_b200 as iq
from test_gpu_window import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _raw(c, Q, out, ws, n_q, window=True):
    lib, st = iq.raw_lib(), torch.cuda.current_stream().cuda_stream
    if not window:
        return lib.isoq_multi_token_attention(c.params.handle, c.cache.c, Q.data_ptr(), iq.ISOQ_BF16, Q.shape[0], n_q,
                                              Q.shape[-2], c.sl.data_ptr(), c.max_len, out.data_ptr(), 0.1,
                                              ws.data_ptr(), ws.numel(), st)
    return lib.isoq_multi_token_attention_window(c.params.handle, c.cache.c, Q.data_ptr(), iq.ISOQ_BF16, Q.shape[0],
                                                 n_q, Q.shape[-2], c.sl.data_ptr(), c.max_len, c.W, c.S,
                                                 out.data_ptr(), iq.ISOQ_F32, 0.1, ws.data_ptr(), ws.numel(), st)


def test_the_longest_chunk_at_d256(oracle):
    """65520 row blocks of 4 fit the grid and are right; one token more is refused, not launched."""
    c = Case([300], 16, 8, 64, 4, n_q=16380, d=256, out="f32", poison=False)
    out = c.run()
    c.Q, out = c.Q[:, -40:].contiguous(), out[:, -40:]
    c.check(oracle, out)
    Q = torch.zeros((1, 16384, 16, 256), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    for window in (True, False):
        assert _raw(c, Q, out, ws, 16384, window) == iq.ISOQ_E_ARG


def test_more_sequences_than_a_grid_holds_are_refused():
    n = 65536
    params = iq.isoq_make_params(0, 128, 1)
    cache = iq.PagedCache(128, 1, 1, torch.zeros((n, 1), dtype=torch.int32))
    x = torch.randn((3, 1, 128), device="cuda")
    i = torch.arange(3, dtype=torch.int32, device="cuda")
    iq.isoq_quantize_append(params, cache, x, x, torch.zeros_like(i), i)
    Q, out = torch.randn((n, 1, 128), device="cuda"), torch.full((n, 1, 128), 3.0, device="cuda")
    lens = torch.full((n,), 3, dtype=torch.int32, device="cuda")
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")

    def calls(m):
        yield lambda: iq.isoq_decode_attention_window(params, cache, Q[:m], lens[:m], 3, 8, 0, out[:m], 0.1, ws)
        yield lambda: iq.isoq_decode_attention(params, cache, Q[:m], lens[:m], 3, out[:m], 0.1, ws)
    for call in calls(n):
        with pytest.raises(iq.IsoqError) as e:
            call()
        assert e.value.code == iq.ISOQ_E_ARG
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())
    for call in calls(n - 1):
        out.fill_(3.0)
        call()
        assert bool((out[:-1] != 3.0).any(-1).all()) and bool((out[-1] == 3.0).all())
    assert iq.isoq_get_status(cache) == 0


@pytest.mark.parametrize("kw", [dict(lens=[32768], hq=32, hkv=4, W=1024, S=4),
                                dict(lens=[9000, 8000], hq=64, hkv=8, W=4096, S=4),
                                dict(lens=[4000, 50], hq=16, hkv=8, W=2000, S=5, d=256),
                                dict(lens=[3000, 0, 777], hq=15, hkv=3, W=777, S=3, bits=4),
                                dict(lens=[40000], hq=4, hkv=1, W=38000, S=4),
                                dict(lens=[900], hq=8, hkv=2, W=300, S=4, n_q=3),
                                dict(lens=[900], hq=8, hkv=2, W=300, S=4, n_q=40),
                                dict(lens=[20000], hq=8, hkv=2, W=16000, S=4, n_q=10)])
def test_a_workspace_of_the_size_asked_for_is_enough(oracle, kw):
    """The bytes behind it stay as they were; one byte less is refused."""
    c = Case(seed=70, **kw)
    n = iq.isoq_window_workspace_bytes(len(c.lens), c.n_q, c.hq, c.hkv, c.d, c.max_len, c.W, c.S)
    raw = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    c.check(oracle, c.run(ws=raw[:n]))
    assert bool((raw[n:] == 0xA5).all())
    with pytest.raises(iq.IsoqError) as e:
        c.run(ws=raw[:n - 1])
    assert e.value.code == iq.ISOQ_E_WORKSPACE


@pytest.mark.parametrize("d,bits,n_q", [(128, 3, 1), (128, 3, 3), (128, 3, 40), (128, 4, 2), (256, 3, 1)])
def test_lengths_next_to_the_largest_position(oracle, d, bits, n_q):
    """Tokens just below 2^31: a length up to 2^31 - 64 is attended as any other, a longer one is
    clamped to that and reported."""
    end, maxp, H, keep = 2 ** 31 - 64, 2 ** 25, 2, 200
    params = iq.isoq_make_params(80, d, H, bits=bits)
    cache = iq.PagedCache(d, H, 8, torch.full((1, maxp), -1, dtype=torch.int32), bits=bits)
    first = (end - keep) // 64
    cache.page_table[0, first:first + 5] = torch.arange(5, dtype=torch.int32, device="cuda").flip(0)
    g = torch.Generator().manual_seed(5)
    pos = torch.arange(end - keep, end + 60, dtype=torch.int64).to(torch.int32)
    K, V = torch.randn((2, len(pos), H, d), generator=g)
    V[keep:] *= 1e3                        # behind the last position that can be attended
    iq.isoq_quantize_append(params, cache, K.cuda(), V.cuda(), torch.zeros(len(pos), dtype=torch.int32, device="cuda"),
                            pos.cuda())
    Q = torch.randn((1, n_q, 8, d), generator=g).cuda()
    W, L = 100, 2 ** 31 - 1
    ws = torch.empty(max(16, iq.isoq_window_workspace_bytes(1, n_q, 8, H, d, L, W, 0)), dtype=torch.uint8, device="cuda")

    def run(n):
        out = torch.full_like(Q, float("nan"))
        iq.isoq_multi_token_attention_window(params, cache, Q, torch.tensor([n], dtype=torch.int32, device="cuda"), L,
                                             W, 0, out, d ** -0.5, ws)
        return out
    want = run(end)
    assert iq.isoq_get_status(cache) == 0
    # the same tokens in a short cache
    short = iq.PagedCache(d, H, 8, torch.arange(5, dtype=torch.int32).flip(0)[None], bits=bits)
    short.blocks.copy_(cache.blocks)
    n = end - first * 64
    other = torch.full_like(Q, float("nan"))
    iq.isoq_multi_token_attention_window(params, short, Q, torch.tensor([n], dtype=torch.int32, device="cuda"), n, W, 0,
                                         other, d ** -0.5, ws if ws.numel() > 1 << 20 else
                                         torch.empty(1 << 22, dtype=torch.uint8, device="cuda"))
    assert bool(torch.isfinite(want).all()) and bool(want.any())
    assert float((want - other).norm() / other.norm()) <= 2 * 5e-4  # each within 5e-4 of the definition
    for n in (end + 1, end + 60, L):
        got = run(n)
        assert iq.isoq_get_status(cache) == iq.ISOQ_ST_LEN_RANGE, n
        iq.isoq_reset_status(cache)
        assert torch.equal(got, want), n
