"""fa2_last_decode_info on the host (no GPU needed)."""
import ctypes
import threading

from attention_fa2_forward_02_gb300 import binding
from attention_fa2_forward_02_gb300 import build as build_mod


def test_a_thread_that_launched_nothing():
    build_mod.build()
    lib, out = binding.library(), {}

    def work():
        out["info"] = binding.fa2_last_decode_info()
        out["null"] = lib.fa2_last_decode_info(ctypes.POINTER(ctypes.c_int32)())

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert out == {"info": -1, "null": 1}  # FA2_ERR_INVALID_ARG
