"""Read-back of cached vectors on the GPU against the plain fp64 reference on the same packed
pages (tests/_window_ref.py), element by element."""
import numpy as np
import pytest
import torch

import rotated_bit_kv_isoquant_b200 as iq
from _window_ref import EPS_HALF, dequantize_pages, window_attention

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


class Store:
    """A cache of sequences in shuffled pages filled by the library's quantiser."""

    def __init__(self, lens, H, d=128, bits=3, rot=0, seed=0, rope=False):
        g = torch.Generator().manual_seed(7000 + seed)
        self.lens, self.H, self.d, self.bits, self.rot, self.seed = lens, H, d, bits, rot, seed
        npg = [-(-n // 64) for n in lens]
        ids = torch.randperm(sum(npg) + 2, generator=g)[:sum(npg)].to(torch.int32)
        self.pt = torch.full((len(lens), max(npg) + 1), -1, dtype=torch.int32)
        for s, n in enumerate(npg):
            self.pt[s, :n] = ids[sum(npg[:s]):sum(npg[:s + 1])]
        self.params = iq.isoq_make_params(seed, d, H, bits=bits, rotation=rot)
        self.cache = iq.PagedCache(d, H, sum(npg) + 2, self.pt, bits=bits)
        self.sid = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).to(torch.int32)
        self.pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)
        scale = torch.exp(torch.empty(2, H, d).uniform_(-2, 2, generator=g))
        K, V = torch.randn((2, len(self.pos), H, d), generator=g) * scale[:, None]
        self.K, self.V = K.cuda(), V.cuda()
        self.table = iq.isoq_rope_table(d, max(lens) + 5) if rope else None
        args = (self.params, self.cache, self.K, self.V, self.sid.cuda(), self.pos.cuda())
        if rope:
            iq.isoq_quantize_append_rope(*args, self.table)
        else:
            iq.isoq_quantize_append(*args)

    def read(self, at, out, rope=False, k=True, v=True, sentinel=float("nan")):
        sid, pos = self.sid[at].cuda(), self.pos[at].cuda()
        K, V = (torch.full((len(at), self.H, self.d), sentinel, dtype=DT[out], device="cuda") if x
                else None for x in (k, v))
        if rope:
            iq.isoq_dequantize_rope(self.params, self.cache, sid, pos, K, V, self.table)
        else:
            iq.isoq_dequantize(self.params, self.cache, sid, pos, K, V)
        return K, V

    def reference(self, oracle, at, out, rope):
        """(K, V) in fp64 and the element bounds.  With S = sum_j |R_ji| |z_j| of an element
        (z = the rotated vector, norm included):
          fp32   (log2 d + 12) 2^-24 S': the levels, the blocks and their four products, the
                 WHT's adds, the factor; S' with the blocks' and the WHT's magnitudes
                 separated, sum_k |M^T z|_k <= 2 S
          bf16   2^-11 S for the rotation as binary16, f16: 2^-21 S for two binary16 parts;
                 both the levels as binary16 (2e-5, 0, 6e-5 of S for 3, 2, 4 bits) and the
                 tensor core's fp32 sums (d 2^-24 S)
          the rope adds the pair's bounds, and 2^-22 of both magnitudes for its own rounding
          half a step of the output type (f16: at least half its smallest subnormal)."""
        p64 = oracle.make_params_v(self.seed, self.d, self.H, self.rot)[1].astype(np.float64)
        blocks = self.cache.blocks.cpu().numpy()
        K, V, kt, vt, R = dequantize_pages(oracle, p64, blocks, self.d, self.bits, self.rot)
        pos = self.pos[at].numpy()
        ph = self.pt[self.sid[at].long(), pos // 64].numpy()
        eL = {2: 0.0, 3: 2e-5, 4: 6e-5}[self.bits]
        e = {"f32": 2 * (np.log2(self.d) + 12) * 2.0 ** -24,
             "bf16": 2.0 ** -11 + eL + self.d * 2.0 ** -24,
             "f16": 2.0 ** -21 + eL + self.d * 2.0 ** -24}[out]
        found = []
        for side, (x, z) in enumerate(((K, kt), (V, vt))):
            x, z = x[ph, pos % 64], z[ph, pos % 64]
            tol = e * np.einsum("nhe,hed->nhd", np.abs(z), np.abs(R))
            if rope and side == 0:
                half = self.d // 2
                ang = pos[:, None, None] * 10000.0 ** (-2.0 * np.arange(half) / self.d)
                a, b = x[..., :half], x[..., half:]
                x = np.concatenate([a * np.cos(ang) + b * np.sin(ang), b * np.cos(ang) - a * np.sin(ang)], -1)
                two = tol[..., :half] + tol[..., half:] + 2.0 ** -22 * (np.abs(a) + np.abs(b))
                tol = np.concatenate([two, two], -1)
            found.append((x, tol + EPS_HALF[out] * np.abs(x) + (2.0 ** -25 if out == "f16" else 0)))
        return found

    def check(self, oracle, at, out, rope=False):
        got = self.read(at, out, rope)
        for name, g, (x, tol) in zip("KV", got, self.reference(oracle, at, out, rope)):
            err = np.abs(g.double().cpu().numpy() - x)
            assert (err <= tol).all(), (name, np.argwhere(~(err <= tol))[:3], np.nanmax(err / tol))
        assert iq.isoq_get_status(self.cache) == 0


FORMATS = [(128, 3, 0), (128, 3, 1), (256, 3, 0), (256, 3, 1), (128, 2, 0), (128, 4, 0), (128, 4, 1)]


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d,bits,rot", FORMATS)
def test_whole_sequences(oracle, d, bits, rot, out):
    s = Store([300, 64, 1, 129], 3, d, bits, rot, seed=d + bits)
    s.check(oracle, torch.arange(len(s.pos)), out)


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d,bits", [(128, 3), (256, 3), (128, 2), (128, 4)])
def test_token_lists(oracle, d, bits, out):
    """Single tokens, runs that begin and end inside pages, any order, the same token twice."""
    s = Store([500, 260], 2, d, bits, seed=3)
    g = torch.Generator().manual_seed(1)
    n = len(s.pos)
    for at in [torch.tensor([0]), torch.tensor([n - 1]), torch.arange(17, 17 + 300), torch.arange(n).flip(0),
               torch.randperm(n, generator=g), torch.tensor([5] * 130 + [700] * 3),
               torch.randint(0, n, (333,), generator=g), torch.arange(0, n, 2), torch.arange(37, 38 + 127)]:
        s.check(oracle, at, out)


@pytest.mark.parametrize("out", ["bf16", "f16"])
@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("d,bits,rot", FORMATS)
def test_long_lists(oracle, d, bits, rot, rope, out):
    """Enough vectors for the tensor-core kernel: runs that start on and off a 16-slot block,
    any order, a ragged end, one side alone."""
    s = Store([1400, 700, 65], 4, d, bits, rot, seed=21, rope=rope)
    g = torch.Generator().manual_seed(5)
    n = len(s.pos)
    for at in [torch.arange(n), torch.arange(3, n - 2), torch.randperm(n, generator=g),
               torch.cat([torch.arange(640, 1300), torch.arange(1400, 1400 + 577), torch.arange(64)])]:
        s.check(oracle, at, out, rope=rope)
    at = torch.cat([torch.arange(n), torch.arange(n)])
    K, V = s.read(at, out, rope)
    assert torch.equal(s.read(at, out, rope, v=False)[0], K) and torch.equal(s.read(at, out, rope, k=False)[1], V)
    sid, pos = s.sid.clone(), s.pos.clone()
    s.sid[7], s.pos[1500], s.pos[n - 1] = 9, -4, 10 ** 6
    bad = s.read(at, out, rope, sentinel=5.0)
    assert iq.isoq_get_status(s.cache) == iq.ISOQ_ST_SEQ_RANGE | iq.ISOQ_ST_POS_RANGE
    keep = torch.ones(n, dtype=torch.bool)
    keep[[7, 1500, n - 1]] = False
    keep = torch.cat([keep, keep]).cuda()
    for got, want in zip(bad, (K, V)):
        assert torch.equal(got[keep], want[keep]) and bool((got[~keep] == 5.0).all())


def test_long_list_into_rows_that_are_not_sector_aligned(oracle):
    """A 16-byte aligned output is enough: the sectors are then written in two halves."""
    s = Store([1400, 700], 4)
    at = torch.arange(2100)
    want = s.read(at, "bf16")
    raw = torch.zeros(2100 * 4 * 128 + 8, dtype=torch.bfloat16, device="cuda")
    K = raw[8:].view(2100, 4, 128)
    assert K.data_ptr() % 32 == 16
    iq.isoq_dequantize(s.params, s.cache, s.sid.cuda(), s.pos.cuda(), K, None)
    assert torch.equal(K, want[0])


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d,bits,H", [(128, 3, 1), (256, 3, 3), (128, 2, 8), (128, 4, 2)])
def test_rope_taken_off(oracle, d, bits, H, out):
    s = Store([700, 90], H, d, bits, seed=11, rope=True)
    s.check(oracle, torch.arange(len(s.pos)), out, rope=True)
    s.check(oracle, torch.randperm(len(s.pos))[:131], out, rope=True)
    s.check(oracle, torch.arange(len(s.pos)), out, rope=False)


def test_one_side_and_an_empty_list():
    s = Store([200], 2)
    at = torch.arange(200)
    K, V = s.read(at, "bf16")
    assert torch.equal(s.read(at, "bf16", v=False)[0], K) and torch.equal(s.read(at, "bf16", k=False)[1], V)
    s.read(at[:0], "bf16")
    assert iq.isoq_get_status(s.cache) == 0


@pytest.mark.parametrize("out,rope", [("bf16", False), ("f32", False), ("bf16", True)])
def test_tokens_out_of_range_are_skipped_and_reported(out, rope):
    s = Store([200, 100], 2, rope=True)
    good = torch.arange(300)
    want = s.read(good, out, rope)
    for sid, pos, bit in [(-1, 0, iq.ISOQ_ST_SEQ_RANGE), (2, 0, iq.ISOQ_ST_SEQ_RANGE), (0, -1, iq.ISOQ_ST_POS_RANGE),
                          (0, 5 * 64, iq.ISOQ_ST_POS_RANGE), (0, 2 ** 31 - 1, iq.ISOQ_ST_POS_RANGE),
                          (1, 2 * 64, iq.ISOQ_ST_PAGE_RANGE)]:
        keep = (s.sid.clone(), s.pos.clone())
        s.sid[77], s.pos[77] = sid, pos
        K, V = s.read(good, out, rope, sentinel=5.0)
        assert iq.isoq_get_status(s.cache) == bit
        iq.isoq_reset_status(s.cache)
        for got, w in ((K, want[0]), (V, want[1])):
            assert bool((got[77] == 5.0).all())
            assert torch.equal(got[:77], w[:77]) and torch.equal(got[78:], w[78:])
        s.sid, s.pos = keep
    # a position past the rotary table
    if rope:
        s.table = s.table[:150].contiguous()
        K, V = s.read(good, out, rope, sentinel=5.0)
        assert iq.isoq_get_status(s.cache) == iq.ISOQ_ST_POS_RANGE
        assert bool((K[150:200] == 5.0).all()) and bool((V[150:200] == 5.0).all())
        assert torch.equal(K[:150], want[0][:150]) and torch.equal(V[200:], want[1][200:])


def test_zero_and_saturated_vectors(oracle):
    s = Store([64], 1)
    s.K.zero_()
    s.V.fill_(60000.0)
    iq.isoq_quantize_append(s.params, s.cache, s.K, s.V, s.sid.cuda(), s.pos.cuda())
    assert iq.isoq_get_status(s.cache) == iq.ISOQ_ST_NORM_SAT
    iq.isoq_reset_status(s.cache)
    s.check(oracle, torch.arange(64), "f32")
    s.check(oracle, torch.arange(64), "bf16")
    assert bool((s.read(torch.arange(64), "bf16")[0] == 0).all())


def test_keys_moved_to_other_positions(oracle):
    """The operators together: keep the sinks and the newest tokens, place them next to each
    other at new positions in another cache, attend them through a window there."""
    d, H, keep = 128, 2, 150
    s = Store([1000], H, d, seed=4, rope=True)
    at = torch.cat([torch.arange(4), torch.arange(1000 - keep, 1000)])
    K, V = s.read(at, "f32", rope=True)
    n = len(at)
    pt = torch.arange(3, dtype=torch.int32).flip(0)[None]
    cache = iq.PagedCache(d, H, 3, pt)
    zero, pos = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")
    iq.isoq_quantize_append_rope(s.params, cache, K, V, zero, pos, s.table)
    Q = torch.randn((1, 8, d), generator=torch.Generator().manual_seed(2)).cuda()
    out = torch.empty_like(Q)
    W, S = 100, 4
    ws = torch.empty(iq.isoq_window_workspace_bytes(1, 1, 8, H, d, n, W, S), dtype=torch.uint8, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    iq.isoq_decode_attention_window(s.params, cache, Q, lens, n, W, S, out, d ** -0.5, ws)
    p64 = oracle.make_params_v(s.seed, d, H, 0)[1].astype(np.float64)
    pages = dequantize_pages(oracle, p64, cache.blocks.cpu().numpy(), d)
    ref, tol = window_attention(pages, pt.numpy(), [n], Q[:, None].cpu().numpy().astype(np.float64),
                                d ** -0.5, W, S)
    assert (np.linalg.norm(out[:, None].cpu().numpy() - ref, axis=-1) <= tol).all()
    # the codes survive the move: V, which has no rotary embedding, is coded as it was
    v_codes = slice(64 * (48 + 2), 64 * (48 + 2 + 48))  # of a block at d = 128, 3 bits
    oldc = oracle.unpack_codes_batch(oracle.v_region_records(np.ascontiguousarray(
        s.cache.blocks.cpu().numpy()[..., v_codes]), d), d)
    newc = oracle.unpack_codes_batch(oracle.v_region_records(np.ascontiguousarray(
        cache.blocks.cpu().numpy()[..., v_codes]), d), d)
    old = oldc[s.pt[0, s.pos[at] // 64].numpy(), :, s.pos[at].numpy() % 64]
    new = newc[pt[0].numpy()[np.arange(n) // 64], :, np.arange(n) % 64]
    assert np.array_equal(old, new)
    assert iq.isoq_get_status(cache) == 0


def test_captured_and_on_another_stream():
    s = Store([500], 4)
    at = torch.arange(500)
    want = s.read(at, "bf16")
    sid, pos = s.sid.cuda(), s.pos.cuda()
    out = [torch.zeros_like(w) for w in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        iq.isoq_dequantize(s.params, s.cache, sid, pos, *out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = s.read(at, "bf16")
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_read_back_refusals():
    s = Store([100], 2)
    lib, st = iq.raw_lib(), torch.cuda.current_stream().cuda_stream
    sid, pos = s.sid.cuda(), s.pos.cuda()
    K = torch.full((100, 2, 128), 3.0, device="cuda")

    def call(**kw):
        a = dict(p=s.params.handle, sid=sid.data_ptr(), pos=pos.data_ptr(), n=100, K=K.data_ptr(), V=None, t=iq.ISOQ_F32)
        a.update(kw)
        return lib.isoq_dequantize(a["p"], s.cache.c, a["sid"], a["pos"], a["n"], a["K"], a["V"], a["t"], st)
    for kw in [dict(p=None), dict(sid=None), dict(pos=None), dict(n=-1), dict(K=None), dict(t=3),
               dict(K=K.data_ptr() + 4), dict(V=K.data_ptr() + 8)]:
        assert call(**kw) == iq.ISOQ_E_ARG, kw
    assert lib.isoq_dequantize_rope(s.params.handle, s.cache.c, sid.data_ptr(), pos.data_ptr(), 100, K.data_ptr(),
                                    None, 0, None, 100, st) == iq.ISOQ_E_ARG
    assert lib.isoq_dequantize_rope(s.params.handle, s.cache.c, sid.data_ptr(), pos.data_ptr(), 100, K.data_ptr(),
                                    None, 0, K.data_ptr(), 0, st) == iq.ISOQ_E_ARG
    other = iq.isoq_make_params(0, 128, 3)
    assert call(p=other.handle) == iq.ISOQ_E_DIM
    torch.cuda.synchronize()
    assert bool((K == 3.0).all()) and call(n=0) == 0
