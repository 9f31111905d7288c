"""The CPython module of the 8-bit operators' calls: other threads run during a call (no GPU needed: the calls are refused)."""
import sys
import threading
import time

import pytest

from weight_only_int4_05_b200 import _lib, build as libbuild


@pytest.mark.parametrize("name,args", [
    ("fp8_quantize", (0x10000, 1, 4, 504, 0x10000, 0x10000, None)),
    ("w8a8_gemm", (0x10000, 0x10000, 0x10000, 0x10000, 0x10000, 1, 4, 8, 504, None)),
    ("w8a8_linear", (0x10000, 1, 0x10000, 0x10000, 0x10000, 4, 8, 504, 0x10000, 16, None)),
    ("moe_route", (0x10000, 3, None, 4, 64, 65, 1, 1, 1, 0, 1.0, 0x10000, 0x10000, None)),
    ("w8a8_moe", (0x10000, 1) + (0x10000,) * 7 + (4, 8, 2, 504, 256, 512, 0x10000, 16, None))])
def test_a_call_lets_other_threads_run(name, args):
    """With a switch interval of minutes nothing but the call itself hands the interpreter over."""
    libbuild.build()
    call = getattr(_lib.calls(), name)
    assert call(*args) == 1
    started, ran = threading.Event(), []
    go = threading.Lock()
    go.acquire()

    def other():
        started.set()
        with go:
            ran.append(True)
    thread = threading.Thread(target=other)
    thread.start()
    started.wait()
    was = sys.getswitchinterval()
    sys.setswitchinterval(600.0)
    try:
        go.release()
        end = time.monotonic() + 30.0
        while not ran and time.monotonic() < end:
            call(*args)
        seen = bool(ran)
    finally:
        sys.setswitchinterval(was)
    thread.join()
    assert seen
