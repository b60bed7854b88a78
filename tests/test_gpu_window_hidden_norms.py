"""A value vector that a query row does not see takes nothing from the row's accuracy, however
large it is and whichever other rows of the call do see it."""
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


def _with_norms(c, norm_of):
    """The case's cache filled again with value vectors of norm norm_of(sequence, position)."""
    n_seqs = len(c.lens)
    sid = torch.repeat_interleave(torch.arange(n_seqs), torch.tensor(c.lens)).to(torch.int32)
    pos = torch.cat([torch.arange(n) for n in c.lens]).to(torch.int32)
    g = torch.Generator().manual_seed(c.seed)
    K, V = torch.randn((2, len(pos), c.hkv, c.d), generator=g)
    norm = torch.tensor([norm_of(int(s), int(p)) for s, p in zip(sid, pos)])
    V *= (norm / c.d ** 0.5)[:, None, None]
    iq.isoq_quantize_append(c.params, c.cache, K.cuda(), V.cuda(), sid.cuda(), pos.cuda())
    c.blocks = c.cache.blocks.cpu().numpy()
    return c


FORMS = [dict(n_q=2), dict(n_q=5), dict(n_q=7, hq=4, hkv=4), dict(n_q=33), dict(n_q=64), dict(n_q=100),
         dict(n_q=3, bits=4), dict(n_q=6, bits=2), dict(n_q=40, bits=4), dict(n_q=70, bits=2), dict(n_q=3, d=256),
         dict(n_q=30, d=256)]


@pytest.mark.parametrize("ratio", [1e4, 1e7])
@pytest.mark.parametrize("where", ["ahead", "behind", "both"])
@pytest.mark.parametrize("i", range(len(FORMS)))
def test_large_values_ahead_of_and_behind_a_row(oracle, i, where, ratio):
    """The chunk's last token, which earlier rows do not see yet, and the first row's first window
    token, which later rows do not see any more, `ratio` times as large as the others."""
    f = dict(hq=8, hkv=2, **FORMS[i]) if "hq" not in FORMS[i] else FORMS[i]
    W, n_q, lens = 90, f["n_q"], [400, 193]
    c = Case(lens, W=W, S=0, out="f32", q="f32", seed=i, poison=False, **f)
    large, small = 3e4, 3e4 / ratio

    def norm_of(s, p):
        ahead, behind = p == lens[s] - 1, p == max(0, lens[s] - n_q - W + 1)
        return large if (ahead and where != "behind") or (behind and where != "ahead") else small
    _with_norms(c, norm_of)
    c.check(oracle, c.run())


@pytest.mark.parametrize("i", range(len(FORMS)))
def test_values_that_grow_along_the_context(oracle, i):
    """Norms from 3e-3 to 3e4 along the positions, with sinks of the largest: every row's own
    largest counts for it."""
    f = dict(hq=8, hkv=2, **FORMS[i]) if "hq" not in FORMS[i] else FORMS[i]
    lens = [400, 150]
    c = Case(lens, W=70, S=0, out="f32", q="f32", seed=30 + i, poison=False, **f)
    _with_norms(c, lambda s, p: 3e-3 * 10.0 ** (7 * p / lens[s]))
    c.check(oracle, c.run())


@pytest.mark.parametrize("i", range(len(FORMS)))
def test_rows_whose_first_values_are_zero(oracle, i):
    """A run of zero vectors first, small ones behind them, a large one that only later rows see."""
    f = dict(hq=8, hkv=2, **FORMS[i]) if "hq" not in FORMS[i] else FORMS[i]
    lens = [300, 170]
    c = Case(lens, W=140, S=3, out="f32", q="f32", seed=60 + i, poison=False, **f)
    _with_norms(c, lambda s, p: 3e4 if p == lens[s] - 1 else 0.0 if p < lens[s] - 110 else 0.01)
    c.check(oracle, c.run())


@pytest.mark.parametrize("where", ["ahead", "behind", "middle"])
@pytest.mark.parametrize("f", [dict(n_q=3, hq=8, hkv=2), dict(n_q=10, hq=8, hkv=2), dict(n_q=70, hq=8, hkv=2),
                               dict(n_q=3, hq=4, hkv=1, bits=4), dict(n_q=2, hq=4, hkv=1, d=256)])
def test_large_values_with_the_window_in_several_chunks(oracle, f, where):
    """The chunks' states meet in the workspace or in a cluster: the rows of each chunk keep
    references of their own."""
    lens, W, n_q = [9000], 8000, f["n_q"]
    c = Case(lens, W=W, S=2, out="f32", q="f32", seed=90, poison=False, **f)
    big = {"ahead": [lens[0] - 1], "behind": [lens[0] - n_q - W + 1], "middle": list(range(4000, 4100))}[where]
    _with_norms(c, lambda s, p: 3e4 if p in big else 3e-3)
    c.check(oracle, c.run())


def test_lifted_rows_repeat_bitwise_and_in_a_graph():
    c = Case([400, 193], 8, 2, 90, 0, n_q=64, out="f32", q="f32", seed=5, poison=False)
    _with_norms(c, lambda s, p: 3e4 if p in (399, 192) else 3e-3)
    want, out, ws = c.run(), torch.empty_like(c.run()), c.workspace()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(ws=ws, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    assert iq.isoq_get_status(c.cache) == 0
