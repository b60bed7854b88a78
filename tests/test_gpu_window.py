"""Sliding-window attention with sinks on the packed cache, on the GPU against the plain
fp64 reference of tests/_window_ref.py on the same packed pages.  Every page slot that no
query of the call may see is poisoned (its norms infinite or NaN, its codes random) and the
page-table entries of the pages in the gap are invalid, so a token that leaks in shows."""
import numpy as np
import pytest
import torch

import rotated_bit_kv_isoquant_b200 as iq
from _window_ref import dequantize_pages, visible, window_attention

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


class Case:
    """A cache of sequences of the given lengths in shuffled pages, filled by the library's
    own quantiser, with what a window (W, S) and n_q query tokens cannot see poisoned."""

    def __init__(self, lens, hq, hkv, W, S, n_q=1, d=128, bits=3, rot=0, q="bf16", out="bf16",
                 seed=0, poison=True, edges=False):
        g = torch.Generator().manual_seed(1000 + seed)
        self.lens, self.hq, self.hkv, self.W, self.S, self.n_q = lens, hq, hkv, W, S, n_q
        self.d, self.bits, self.rot, self.out_t, self.seed = d, bits, rot, out, seed
        n_seqs, npg = len(lens), [-(-n // 64) for n in lens]
        maxp, total = max(1, max(npg)), sum(npg) + 1
        ids = torch.randperm(total, generator=g)[:sum(npg)].to(torch.int32)
        self.pt = torch.full((n_seqs, maxp), -1, dtype=torch.int32)
        o = 0
        for s, n in enumerate(npg):
            self.pt[s, :n] = ids[o:o + n]
            o += n
        self.params = iq.isoq_make_params(seed, d, hkv, bits=bits, rotation=rot)
        self.cache = iq.PagedCache(d, hkv, total, self.pt, bits=bits)
        sid = torch.repeat_interleave(torch.arange(n_seqs), torch.tensor(lens)).to(torch.int32)
        pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)
        scale = torch.exp(torch.empty(2, hkv, d).uniform_(-2, 2, generator=g))
        K, V = torch.randn((2, len(pos), hkv, d), generator=g) * scale[:, None]
        if edges:  # the outermost visible tokens weigh most: losing one shows
            for s, n in enumerate(lens):
                ends = {e for i in range(n_q) for t in [visible(n - n_q + i, W, S)]
                        for e in [*t[:1], *t[-1:], S - 1, n - n_q + i + 1 - W] if 0 <= e < n}
                V[(sid == s) & torch.isin(pos, torch.tensor(sorted(int(e) for e in ends)))] *= 50
        if len(pos):
            iq.isoq_quantize_append(self.params, self.cache, K.to(torch.bfloat16).cuda(),
                                    V.to(torch.bfloat16).cuda(), sid.cuda(), pos.cuda())
        self.call_pt = self.pt.clone()
        blocks = self.cache.blocks.cpu().numpy()
        if poison:
            rng = np.random.default_rng(seed)
            cb = bits * d // 8
            bad = np.array([0x7c00, 0xfc00, 0x7e00, 0x7bff], np.uint16)  # inf, -inf, NaN, max
            seen = np.zeros((total, 64), bool)
            for s, n in enumerate(lens):
                for i in range(n_q):
                    t = visible(n - n_q + i, W, S)
                    seen[self.pt[s, t // 64].numpy(), t % 64] = True
            for off in (64 * cb, 64 * (2 * cb + 2)):
                nv = blocks[..., off:off + 128].copy().view(np.uint16)
                nv = np.where(seen[:, None], nv, rng.choice(bad, nv.shape))
                blocks[..., off:off + 128] = nv.view(np.uint8)
            self.cache.blocks.copy_(torch.from_numpy(blocks))
            for s in range(n_seqs):
                for p in range(maxp):
                    ph = int(self.pt[s, p])
                    if ph >= 0 and not seen[ph].any():
                        self.call_pt[s, p] = [-1, 2 ** 31 - 1, -2 ** 31][p % 3]
            self.cache.page_table.copy_(self.call_pt)
        self.blocks = blocks
        self.Q = torch.randn((n_seqs, n_q, hq, d), generator=g).to(DT[q]).cuda()
        self.sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.max_len = max(lens)

    def workspace(self, fill=0xFF):
        n = iq.isoq_window_workspace_bytes(len(self.lens), self.n_q, self.hq, self.hkv, self.d,
                                           self.max_len, self.W, self.S)
        return torch.full((max(n, 16),), fill, dtype=torch.uint8, device="cuda")

    def run(self, chunk=None, ws=None, out=None):
        chunk = self.n_q > 1 if chunk is None else chunk
        Q = self.Q if chunk else self.Q[:, 0].contiguous()
        out = torch.full(Q.shape, float("nan"), dtype=DT[self.out_t], device="cuda") if out is None else out
        call = iq.isoq_multi_token_attention_window if chunk else iq.isoq_decode_attention_window
        call(self.params, self.cache, Q, self.sl, self.max_len, self.W, self.S, out,
             self.d ** -0.5, self.workspace() if ws is None else ws)
        return out

    def check(self, oracle, out):
        p64 = oracle.make_params_v(self.seed, self.d, self.hkv, self.rot)[1].astype(np.float64)
        pages = dequantize_pages(oracle, p64, self.blocks, self.d, self.bits, self.rot)
        ref, tol = window_attention(pages, self.pt.numpy(), self.lens,
                                    self.Q.float().cpu().numpy().astype(np.float64),
                                    self.d ** -0.5, self.W, self.S, self.bits, self.out_t)
        got = out.float().cpu().numpy().astype(np.float64).reshape(ref.shape)
        assert np.isfinite(got).all()
        err = np.linalg.norm(got - ref, axis=-1)
        assert (err <= tol).all(), f"worst {np.max(err - tol)}, {np.argwhere(err > tol)[:4]}"
        assert iq.isoq_get_status(self.cache) == 0


def _case(seed, **kw):
    return Case(seed=seed, **kw)


DECODE = [
    dict(lens=[1], hq=4, hkv=1, W=1, S=0),
    dict(lens=[0, 1, 2, 63, 64, 65, 129], hq=8, hkv=2, W=64, S=0),
    dict(lens=[300, 0, 77, 1000], hq=8, hkv=2, W=100, S=4),
    dict(lens=[1000, 640], hq=32, hkv=4, W=64, S=64, out="f32"),
    dict(lens=[1000, 641], hq=32, hkv=4, W=65, S=65, q="f16", out="f16"),
    dict(lens=[700], hq=15, hkv=3, W=10 ** 9, S=3, q="f32"),             # the whole context
    dict(lens=[700, 90], hq=16, hkv=1, W=1, S=1),
    dict(lens=[700, 90], hq=7, hkv=7, W=200, S=10 ** 9),                 # sinks past the context
    dict(lens=[2500, 1800, 64], hq=16, hkv=8, W=777, S=5, d=256),
    dict(lens=[2500, 30], hq=8, hkv=2, W=130, S=100, d=256, rot=1, out="f16"),
    dict(lens=[500, 0, 900], hq=12, hkv=3, W=250, S=3, bits=4, q="f32"),
    dict(lens=[500, 1, 900], hq=12, hkv=3, W=250, S=70, bits=2, rot=1),
    dict(lens=[5000, 4700, 4999], hq=64, hkv=8, W=4096, S=4),
    dict(lens=[9000], hq=8, hkv=1, W=8192, S=0, out="f16"),
    # more (sequence, KV head) units than SMs, chunks as clusters of 4-warp CTAs or one CTA each
    dict(lens=list(range(0, 1200, 30)), hq=32, hkv=8, W=700, S=4),
    dict(lens=list(range(5, 645, 16)), hq=15, hkv=5, W=300, S=70, bits=4, out="f16"),
    dict(lens=list(range(0, 1400, 70)), hq=16, hkv=8, W=900, S=1, d=256),
    # few units and a long window: partial results and the combine
    dict(lens=[40000], hq=4, hkv=1, W=38000, S=4),
    dict(lens=[33000, 10], hq=2, hkv=1, W=32000, S=0, bits=2, out="f16"),
    dict(lens=[30000], hq=2, hkv=1, W=29999, S=1, d=256, out="f32"),
]


@pytest.mark.parametrize("i", range(len(DECODE)))
def test_decode_window(oracle, i):
    c = _case(i, **DECODE[i])
    c.check(oracle, c.run())


@pytest.mark.parametrize("W,S", [(1, 0), (2, 1), (63, 3), (64, 64), (65, 5), (128, 0), (129, 63)])
@pytest.mark.parametrize("n_q", [1, 3, 40])
def test_window_edges(oracle, W, S, n_q):
    """The first and last visible tokens carry the weight, everything next to them is poison."""
    c = _case(W, lens=[400, 193, 128, 39], hq=8, hkv=2, W=W, S=S, n_q=n_q, edges=True, out="f32")
    c.check(oracle, c.run())


CHUNK = [
    dict(lens=[300, 5, 0, 64], hq=8, hkv=2, W=100, S=4, n_q=2),          # rows before position 0
    dict(lens=[300, 129], hq=8, hkv=2, W=1, S=0, n_q=3),
    dict(lens=[1000, 650], hq=8, hkv=2, W=200, S=70, n_q=7),             # 28 rows per KV head
    dict(lens=[1000, 20], hq=32, hkv=4, W=128, S=0, n_q=16, q="f16", out="f16"),  # 128 rows
    dict(lens=[900, 300], hq=32, hkv=8, W=64, S=5, n_q=129),             # window shorter than the chunk
    dict(lens=[900], hq=64, hkv=8, W=10 ** 9, S=0, n_q=33, out="f32"),   # the whole context
    dict(lens=[600, 100], hq=5, hkv=5, W=90, S=3, n_q=131, q="f32"),     # one row per token
    dict(lens=[600, 300], hq=12, hkv=3, W=100, S=3, n_q=5, bits=4),
    dict(lens=[600, 300], hq=12, hkv=3, W=100, S=65, n_q=50, bits=4, rot=1),
    dict(lens=[600, 300], hq=12, hkv=3, W=100, S=3, n_q=9, bits=2),
    dict(lens=[600, 300], hq=12, hkv=3, W=100, S=3, n_q=3, bits=2),
    dict(lens=[600, 300], hq=8, hkv=2, W=100, S=3, n_q=70, bits=2, out="f16"),
    dict(lens=[900, 130], hq=16, hkv=8, W=300, S=5, n_q=11, d=256),
    dict(lens=[4400], hq=8, hkv=1, W=3000, S=64, n_q=200),
    # 36 .. 128 rows per KV head: two halves take the pages in turn (one page, two, odd and even)
    dict(lens=[40, 64, 65, 128, 130, 200], hq=8, hkv=2, W=10 ** 6, S=0, n_q=9, out="f32"),
    dict(lens=[3000, 61, 0, 2], hq=8, hkv=2, W=500, S=3, n_q=32, q="f16", out="f16"),
    # 129 rows and more: two row blocks share the pages, the second one short or empty
    dict(lens=[700, 64, 3], hq=3, hkv=3, W=300, S=5, n_q=129, out="f32"),
    dict(lens=[700, 100], hq=16, hkv=2, W=130, S=64, n_q=33),
    dict(lens=[2000, 320], hq=8, hkv=1, W=600, S=1, n_q=64, bits=4, q="f16", out="f16"),
    dict(lens=[64], hq=16, hkv=1, W=7, S=0, n_q=64, bits=2),             # one page
    dict(lens=[20000], hq=8, hkv=2, W=16000, S=4, n_q=10, out="f32"),    # chunks and the combine
    dict(lens=[20000, 9000], hq=8, hkv=2, W=16000, S=4, n_q=70),
]


@pytest.mark.parametrize("i", range(len(CHUNK)))
def test_chunk_window(oracle, i):
    c = _case(50 + i, **CHUNK[i])
    c.check(oracle, c.run())


@pytest.mark.parametrize("n_q,hq,hkv,d", [(1, 8, 2, 128), (1, 4, 2, 256), (3, 8, 2, 128), (40, 8, 2, 128), (200, 8, 2, 128),
                                         (9, 4, 2, 256)])
def test_empty_sequences_give_zeros(n_q, hq, hkv, d):
    c = _case(1, lens=[0, 0, 0], hq=hq, hkv=hkv, W=5, S=2, n_q=n_q, d=d)
    assert c.max_len == 0 and bool((c.run() == 0).all())
    c.max_len, c.W = 10 ** 6, 10 ** 6      # a plan of many chunks, all of them empty
    assert bool((c.run() == 0).all()) and iq.isoq_get_status(c.cache) == 0


def test_a_long_chunk_at_d256(oracle):
    c = _case(2, lens=[700, 150], hq=4, hkv=2, W=120, S=3, n_q=150, d=256)
    c.check(oracle, c.run())


def test_sequences_that_share_pages(oracle):
    """A shared prefix: three sequences whose first pages are the same physical pages."""
    c = _case(3, lens=[500, 500, 500], hq=8, hkv=2, W=200, S=64, poison=False)
    c.pt[1:, :5] = c.pt[0, :5]
    c.cache.page_table.copy_(c.pt)
    c.check(oracle, c.run())


def test_two_streams_at_once():
    a = _case(4, lens=[3000, 2000], hq=32, hkv=4, W=1500, S=4)
    b = _case(5, lens=[900, 1000], hq=64, hkv=8, W=700, S=64, n_q=40)
    want = a.run(), b.run()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    ws, out = (a.workspace(), b.workspace()), (torch.empty_like(want[0]), torch.empty_like(want[1]))
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(sa):
            a.run(ws=ws[0], out=out[0])
        with torch.cuda.stream(sb):
            b.run(ws=ws[1], out=out[1])
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


FIRST_CAPTURED = """
import torch, rotated_bit_kv_isoquant_b200 as iq
d, H, L = 128, 2, 1500
p = iq.isoq_make_params(0, d, H)
c = iq.PagedCache(d, H, 24, torch.arange(24)[None])
x = torch.randn(L, H, d, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
sid, pos = torch.zeros(L, dtype=torch.int32, device="cuda"), torch.arange(L, dtype=torch.int32, device="cuda")
iq.isoq_quantize_append(p, c, x, x, sid, pos)
lens = torch.tensor([L], dtype=torch.int32, device="cuda")
for n_q in (1, 4, 50):
    Q = torch.randn(1, n_q, 8, d, device="cuda")
    out, again = torch.zeros(2, 1, n_q, 8, d, device="cuda")
    ws = torch.empty(max(16, iq.isoq_window_workspace_bytes(1, n_q, 8, H, d, L, 700, 4)), dtype=torch.uint8, device="cuda")
    run = lambda o: iq.isoq_multi_token_attention_window(p, c, Q, lens, L, 700, 4, o, 0.1, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(out)
    g.replay()
    run(again)
    torch.cuda.synchronize()
    assert torch.equal(out, again) and bool(out.any()), n_q
K = torch.zeros(L, H, d, dtype=torch.bfloat16, device="cuda")
for n in (5, L):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        iq.isoq_dequantize(p, c, sid[:n], pos[:n], K[:n], None)
    g.replay()
    torch.cuda.synchronize()
    assert bool(K[n - 1].any())
assert iq.isoq_get_status(c) == 0
print("ok")
"""


def test_the_first_call_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", FIRST_CAPTURED], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr[-2000:]


def test_one_token_chunk_is_the_decode(oracle):
    c = _case(3, lens=[500, 90], hq=8, hkv=2, W=100, S=4)
    a, b = c.run(chunk=False), c.run(chunk=True)
    assert torch.equal(a, b[:, 0])


def test_open_window_matches_the_whole_context_calls():
    """A window of at least the context, fp32 out: the plain decode's arithmetic on the same
    tokens (both within the decode's documented error of the same sums)."""
    c = _case(4, lens=[3000, 1777], hq=32, hkv=4, W=2 ** 31 - 1, S=0, out="f32", poison=False)
    a = c.run()
    n = iq.isoq_decode_workspace_bytes(2, 32, 4, 128, 3000)
    ws = torch.empty((n,), dtype=torch.uint8, device="cuda")
    b = torch.empty_like(a)
    iq.isoq_decode_attention(c.params, c.cache, c.Q[:, 0].contiguous(), c.sl, 3000, b, 128 ** -0.5, ws)
    err = (a - b).norm(dim=-1) / b.norm(dim=-1)
    assert float(err.max()) <= 2 * 5e-4  # each is within 5e-4 of the definition


def test_a_step_with_its_window(oracle):
    """The operators as a server uses them: append a token, attend through the window, with
    pages recycled as the window passes them; two steps captured into one graph and replayed."""
    c = _case(5, lens=[640, 700], hq=8, hkv=2, W=128, S=4, out="f32", poison=False)
    d, H = 128, 2
    g = torch.Generator().manual_seed(9)
    K, V = (torch.randn((2, 2, H, d), generator=g) * 2).to(torch.bfloat16).cuda()
    sid = torch.arange(2, dtype=torch.int32, device="cuda")
    pos = c.sl - 1
    ws, out = c.workspace(), torch.empty((2, 8, d), device="cuda")
    Q = c.Q[:, 0].contiguous()

    def step():
        iq.isoq_quantize_append(c.params, c.cache, K, V, sid, pos)
        iq.isoq_decode_attention_window(c.params, c.cache, Q, c.sl, c.max_len, c.W, c.S, out,
                                        d ** -0.5, ws)
    step()
    eager = out.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    out.zero_()
    ws.fill_(0xFF)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    c.blocks = c.cache.blocks.cpu().numpy()
    c.check(oracle, out[:, None])
    # lengths change between replays: the graph reads them from the device
    c.sl -= 70
    c.lens = [570, 630]
    graph.replay()
    torch.cuda.synchronize()
    c.sl += 70
    c.blocks = c.cache.blocks.cpu().numpy()
    c.check(oracle, out[:, None])


def test_calls_repeat_bitwise_and_on_another_stream():
    c = _case(6, lens=[5000, 3000, 64], hq=32, hkv=8, W=2048, S=64)
    a = c.run()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        b = c.run()
    torch.cuda.current_stream().wait_stream(stream)
    assert torch.equal(a, b) and torch.equal(a, c.run(ws=c.workspace(fill=0)))


def test_rows_behind_the_last_sequence_stay_as_they_were():
    c = _case(7, lens=[300, 200, 100], hq=8, hkv=2, W=64, S=4)
    out = torch.full((3, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lib, Q = iq.raw_lib(), c.Q[:, 0].contiguous()
    ws = c.workspace()
    rc = lib.isoq_decode_attention_window(c.params.handle, c.cache.c, Q.data_ptr(), iq.ISOQ_BF16, 2, 8,
                                          c.sl.data_ptr(), 300, 64, 4, out.data_ptr(), iq.ISOQ_BF16,
                                          128 ** -0.5, ws.data_ptr(), ws.numel(),
                                          torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    want = c.run()
    assert torch.equal(out[:2], want[:2]) and bool((out[2] == 7.0).all())


def test_lengths_beyond_the_bounds_are_clamped_and_reported(oracle):
    c = _case(8, lens=[300, 200], hq=8, hkv=2, W=64, S=4, poison=False, out="f32")
    want = c.run()
    c.max_len, c.lens = 250, [250, 200]   # the plan's bound below a length on the device
    got = c.run()
    assert iq.isoq_get_status(c.cache) == iq.ISOQ_ST_LEN_RANGE
    iq.isoq_reset_status(c.cache)
    c.check(oracle, got)
    assert torch.equal(got[1], want[1])
    c.max_len = 10 ** 6
    c.sl.copy_(torch.tensor([2 ** 31 - 1, -2 ** 31], dtype=torch.int32))
    got = c.run()
    assert iq.isoq_get_status(c.cache) == iq.ISOQ_ST_LEN_RANGE
    iq.isoq_reset_status(c.cache)
    c.lens = [320, 0]                     # the page table's end; a negative length is empty
    assert bool((got[1] == 0).all()) and bool(torch.isfinite(got).all())


def test_a_page_out_of_range_is_skipped_and_reported():
    c = _case(9, lens=[300], hq=8, hkv=2, W=128, S=4, poison=False)
    c.cache.page_table[0, 3] = 10 ** 6
    out = c.run()
    assert iq.isoq_get_status(c.cache) == iq.ISOQ_ST_PAGE_RANGE
    assert bool(torch.isfinite(out).all())


def test_window_refusals():
    c = _case(10, lens=[100], hq=8, hkv=2, W=64, S=4)
    Q, out, ws = c.Q[:, 0].contiguous(), torch.full((1, 8, 128), 3.0, device="cuda"), c.workspace()
    lib, st = iq.raw_lib(), torch.cuda.current_stream().cuda_stream

    def call(**kw):
        a = dict(params=c.params.handle, Q=Q.data_ptr(), q=iq.ISOQ_BF16, n=1, hq=8,
                 sl=c.sl.data_ptr(), L=100, W=64, S=4, out=out.data_ptr(), t=iq.ISOQ_F32,
                 scale=0.1, ws=ws.data_ptr(), nb=ws.numel())
        a.update(kw)
        return lib.isoq_decode_attention_window(a["params"], c.cache.c, a["Q"], a["q"], a["n"], a["hq"],
                                                a["sl"], a["L"], a["W"], a["S"], a["out"], a["t"],
                                                a["scale"], a["ws"], a["nb"], st)
    for kw, want in [(dict(W=0), iq.ISOQ_E_ARG), (dict(W=-5), iq.ISOQ_E_ARG), (dict(S=-1), iq.ISOQ_E_ARG),
                     (dict(t=3), iq.ISOQ_E_ARG), (dict(q=-1), iq.ISOQ_E_ARG), (dict(out=None), iq.ISOQ_E_ARG),
                     (dict(Q=None), iq.ISOQ_E_ARG), (dict(sl=None), iq.ISOQ_E_ARG), (dict(ws=None), iq.ISOQ_E_ARG),
                     (dict(L=-1), iq.ISOQ_E_ARG), (dict(n=2), iq.ISOQ_E_ARG), (dict(hq=7), iq.ISOQ_E_GQA),
                     (dict(hq=34), iq.ISOQ_E_GQA), (dict(nb=8), iq.ISOQ_E_WORKSPACE),
                     (dict(ws=ws.data_ptr() + 4), iq.ISOQ_E_WORKSPACE),
                     (dict(out=out.data_ptr() + 8), iq.ISOQ_E_ARG), (dict(Q=Q.data_ptr() + 2), iq.ISOQ_E_ARG), (dict(scale=float("nan")), iq.ISOQ_E_ARG)]:
        assert call(**kw) == want, kw
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())
    assert call(n=0) == 0 and bool((out == 3.0).all())
