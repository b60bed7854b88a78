"""What a read-back reports and leaves alone when listed tokens are out of range, for every
choice of outputs (either of K and V may be absent), on short and on long lists."""
import pytest
import torch

import rotated_bit_kv_isoquant_b200 as iq
from test_gpu_dequantize import Store

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


@pytest.mark.parametrize("k,v", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("d,out", [(128, "bf16"), (128, "f16"), (256, "bf16"), (256, "f16"), (128, "f32")])
def test_every_bad_token_is_reported_whichever_outputs_are_given(d, out, rope, k, v):
    s = Store([1400, 700, 65], 4, d, seed=31, rope=True)
    n = len(s.pos)
    assert n * 4 * 128 >= 2 ** 20     # one side alone is a long list as well
    bad = [(9, 0, iq.ISOQ_ST_SEQ_RANGE), (-1, 0, iq.ISOQ_ST_SEQ_RANGE), (0, -4, iq.ISOQ_ST_POS_RANGE),
           (0, 10 ** 6, iq.ISOQ_ST_POS_RANGE), (2, 3 * 64, iq.ISOQ_ST_PAGE_RANGE)]
    if rope:
        bad.append((0, s.table.shape[0], iq.ISOQ_ST_POS_RANGE))  # a position past the rotary table
    sid, pos = s.sid.clone(), s.pos.clone()
    for count in (n, 40):
        at = torch.arange(count)
        want = s.read(at, out, rope, k=k, v=v)
        assert iq.isoq_get_status(s.cache) == 0
        for bad_sid, bad_pos, bit in bad:
            for i in (7, 39, count - 1):
                s.sid[i], s.pos[i] = bad_sid, bad_pos
                got = s.read(at, out, rope, k=k, v=v, sentinel=5.0)
                assert iq.isoq_get_status(s.cache) == bit, (count, i, bad_sid, bad_pos)
                iq.isoq_reset_status(s.cache)
                for g, w in zip(got, want):
                    if w is not None:
                        assert bool((g[i] == 5.0).all())
                        assert torch.equal(g[:i], w[:i]) and torch.equal(g[i + 1:], w[i + 1:])
                s.sid.copy_(sid)
                s.pos.copy_(pos)
