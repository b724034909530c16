"""The extension module through which Python calls the packed-sequence operators, on the CPU: its
entry points are replaced by functions of the test's own, its tensors by objects that answer what
it asks of a tensor."""
import ctypes
import importlib
import math
import subprocess
import threading
import time

import pytest

F32, BF16, I32 = object(), object(), object()
NAMES = ("rr_qk_norm_rope_fwd", "rr_qk_norm_rope_bwd", "rr_attention_packed_fwd",
         "rr_attention_packed_bwd", "rr_token_logprob_fwd", "rr_token_logprob_bwd")


class Fake:
    """What the module asks of a tensor."""

    def __init__(self, dtype, *shape, address=64):
        self.dtype, self.shape, self.address = dtype, tuple(shape), address

    def stride(self):
        return tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.address

    def get_device(self):
        return 0

    @property
    def nbytes(self):
        return math.prod(self.shape)


@pytest.fixture()
def slow(tmp_path):
    """The module with an entry point that takes 0.3 s for each of its six."""
    import __graft_entry__
    import row_reduction_pass_gb300.rr as rr
    __graft_entry__.build()
    module = importlib.import_module("row_reduction_pass_gb300._call")
    src, lib = tmp_path / "slow.c", tmp_path / "slow.so"
    src.write_text("#include <time.h>\nint slow(void) {\n"
                   "  struct timespec t = {0, 300000000};\n  return nanosleep(&t, 0) ? 1 : 7;\n}\n")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(lib), str(src)], check=True)
    entry = ctypes.cast(ctypes.CDLL(str(lib)).slow, ctypes.c_void_p).value
    module.setup(F32, BF16, I32, lambda: 0, lambda device: 0, (entry,) * len(NAMES))
    yield module
    rr._calls = None  # (set up again at the next call)


def calls(m):
    q, k, w = Fake(BF16, 5, 4, 64), Fake(BF16, 5, 2, 64), Fake(BF16, 64)
    tab, pos, cu = Fake(F32, 9, 32), Fake(I32, 5), Fake(I32, 3)
    lse, x, row = Fake(F32, 4, 5), Fake(F32, 5, 7), Fake(F32, 5)
    ws = Fake(F32, 100)
    return {
        "rope_fwd": lambda: m.rope_fwd(q, k, w, w, tab, tab, pos, q, k, 1e-6, False, None, 0),
        "rope_bwd": lambda: m.rope_bwd(q, k, q, k, w, w, tab, tab, pos, q, k, w, w, 1e-6, False,
                                       ws, None, 0),
        "attn_fwd": lambda: m.attn_fwd(q, k, k, cu, q, lse, 0.1, 0),
        "attn_bwd": lambda: m.attn_bwd(q, q, k, k, q, lse, cu, q, k, k, 0.1, ws, 0),
        "logprob_fwd": lambda: m.logprob_fwd(x, pos, row, None, None, None, None, None, None, 1.0,
                                             -100, None, 0),
        "logprob_bwd": lambda: m.logprob_bwd(x, pos, row, row, row, x, None, None, 1.0, -100, 0)}


@pytest.mark.parametrize("name", ["rope_fwd", "rope_bwd", "attn_fwd", "attn_bwd", "logprob_fwd",
                                  "logprob_bwd"])
def test_other_threads_run_during_a_call(slow, name):
    """A thread that wakes every 5 ms does so during a call of 300 ms (at least 3 times, however
    busy the machine)."""
    call, ticks, done = calls(slow)[name], [], threading.Event()

    def tick():
        while not done.is_set():
            ticks.append(time.monotonic())
            time.sleep(0.005)

    thread = threading.Thread(target=tick)
    thread.start()
    try:
        while not ticks:
            time.sleep(0.001)
        begin = time.monotonic()
        assert call() == 7
        end = time.monotonic()
    finally:
        done.set()
        thread.join()
    assert end - begin >= 0.29
    assert sum(begin + 0.02 < t < end - 0.02 for t in ticks) >= 3
