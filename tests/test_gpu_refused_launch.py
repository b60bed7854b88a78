"""A launch that the CUDA runtime refuses is reported by the call's return value and leaves no
error behind: the caller's next check of the thread's last error is about its own work.

The refusal is made on the host: work on a stream whose capture has been invalidated (by a
synchronisation, which a capturing stream does not allow) is turned down before anything is
launched."""
import ctypes
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import rotated_bit_kv_isoquant_b200 as iq
from test_gpu_window import Case

pytestmark = pytest.mark.gpu
CAPTURE_INVALIDATED = 901  # cudaErrorStreamCaptureInvalidated


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _calls(c):
    """Every attention and read-back call on the case's cache, by the kernel behind it."""
    lib, d = iq.raw_lib(), c.d
    out = torch.zeros((c.n_q, c.hq, d), device="cuda")
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    Q, n_seqs = c.Q, len(c.lens)
    keep = [out, ws, Q]

    def window(n_q):
        return lambda st: lib.isoq_multi_token_attention_window(
            c.params.handle, c.cache.c, Q.data_ptr(), iq.ISOQ_BF16, n_seqs, n_q, c.hq, c.sl.data_ptr(), c.max_len,
            c.W, c.S, out.data_ptr(), iq.ISOQ_F32, 0.1, ws.data_ptr(), ws.numel(), st)

    def whole(n_q):
        return lambda st: lib.isoq_multi_token_attention(
            c.params.handle, c.cache.c, Q.data_ptr(), iq.ISOQ_BF16, n_seqs, n_q, c.hq, c.sl.data_ptr(), c.max_len,
            out.data_ptr(), 0.1, ws.data_ptr(), ws.numel(), st)

    i = torch.zeros(40, dtype=torch.int32, device="cuda")
    K = torch.zeros((40, c.hkv, d), device="cuda")
    keep += [i, K]

    def read(st):
        return lib.isoq_dequantize(c.params.handle, c.cache.c, i.data_ptr(), i.data_ptr(), 40, K.data_ptr(), None,
                                   iq.ISOQ_F32, st)
    return [window(1), window(2), window(c.n_q), whole(1), whole(2), whole(c.n_q), read], keep


@pytest.mark.parametrize("bits", [3, 4])
def test_a_refused_launch_leaves_no_error_behind(bits):
    # in a thread of its own: isoq_last_cuda_error, which is the thread's, is left set
    with ThreadPoolExecutor(1) as pool:
        pool.submit(_refuse_each, bits).result()


def _refuse_each(bits):
    c = Case([300], 8, 2, 100, 4, n_q=40, bits=bits, seed=3, poison=False)
    calls, keep = _calls(c)
    rt = ctypes.CDLL("libcudart.so.12")  # the runtime that the library and torch share
    good = torch.cuda.current_stream().cuda_stream
    for call in calls:                   # each call is a good one on an ordinary stream
        assert call(good) == 0
    torch.cuda.synchronize()
    for call in calls:
        stream = torch.cuda.Stream()
        st, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
        assert rt.cudaStreamBeginCapture(st, 2) == 0
        assert rt.cudaStreamSynchronize(st) != 0          # not while capturing: the capture is void
        rt.cudaGetLastError()
        assert call(stream.cuda_stream) == iq.ISOQ_E_CUDA
        assert iq.raw_lib().isoq_last_cuda_error() == CAPTURE_INVALIDATED
        left = rt.cudaPeekAtLastError()
        assert rt.cudaStreamEndCapture(st, ctypes.byref(graph)) != 0
        rt.cudaGetLastError()
        assert left == 0
        assert call(good) == 0
    torch.cuda.synchronize()
    assert iq.isoq_get_status(c.cache) == 0
    del keep
