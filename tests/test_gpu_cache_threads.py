"""The cache's calls through the CPython module leave other Python threads running, as the calls
through ctypes do: here with entry points in the library's places that take their time on the host."""
import ctypes
import subprocess
import threading
import time

import pytest
import torch

from cache_ref import DEV
from parity import say

from gated_delta_rule_81_amd import _lib

SLOW = """
#include <unistd.h>
long quick(void) { return 0; }
int slow(void) { usleep(400000); return 0; }
"""


@pytest.mark.gpu
def test_other_threads_run_meanwhile(tmp_path):
    src, path = tmp_path / "slow.c", tmp_path / "slow.so"
    src.write_text(SLOW)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-o", str(path), str(src)], check=True)
    handle = ctypes.CDLL(str(path))
    address = lambda lib, name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
    m, own = _lib.cache_calls(), _lib.lib()
    z = lambda *s: torch.zeros(*s, device=DEV)
    i = lambda *s: z(*s).int()
    k, cache, table, lens = z(4, 2, 64), z(9, 16, 2, 64), i(4, 3), i(4)
    torch.cuda.synchronize()
    append = lambda: m.append(0, k, k, cache, cache, table, lens, None, None, None, None, 0, False)
    attend = lambda: m.attention(0, k, cache, cache, table, lens, None, None, None, 0.125, 64, True)
    ticks, stop = [0], threading.Event()

    def count():
        while not stop.is_set():
            ticks[0] += 1
            time.sleep(0.001)

    thread = threading.Thread(target=count)
    try:
        m.bind(address(handle, "slow"), address(handle, "slow"), address(handle, "quick"))
        thread.start()
        for name, call in (("append", append), ("attention", attend)):
            say("the module and other threads", name)
            before, t0 = ticks[0], time.monotonic()
            done = call()
            took = time.monotonic() - t0
            assert done is not None and done[0] == 0 and took > 0.39
            assert ticks[0] - before > 20, name  # of some 300; one or two with the lock held
    finally:
        stop.set()
        if thread.is_alive():
            thread.join()
        m.bind(*(address(own, n) for n in ("kda_cache_append", "kda_prefix_attn_fwd",
                                           "kda_prefix_attn_workspace_size")))
