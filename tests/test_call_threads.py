"""The compiled check-and-call beside other Python threads."""
import ctypes
import os
import threading

import pytest
import torch

from test_call_checks import LIB, NAMES, buffers, result

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not os.path.exists(LIB), reason="libmi355moe.so not built")]
DEV = "cuda"


@pytest.fixture(scope="module")
def m():
    import mxfp8_mxfp4_experts_amd as m
    return m


@pytest.mark.parametrize("name", NAMES)
def test_other_threads_run_during_the_call(m, name):
    """The helper gives the interpreter's lock up before it calls: in the C function's place stands
    the one that says whether the calling thread holds it."""
    from mxfp8_mxfp4_experts_amd import _binding as B
    from mxfp8_mxfp4_experts_amd import _tensor_args as ck
    holds = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    assert getattr(ck, name)(holds, B._raw_stream, *buffers(m)[name].values()) == 0


def test_threads_with_streams_of_their_own(m):
    """Every call from four threads at once, each on its stream and in its buffers."""
    want = {s: {n: result(getattr(m, "moe_" + n)(**kw)) for n, kw in buffers(m, s).items()}
            for s in range(4)}
    sets = {s: buffers(m, s) for s in range(4)}
    torch.cuda.synchronize()
    wrong = []

    def run(s):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    for n, kw in sets[s].items():
                        got = result(getattr(m, "moe_" + n)(**kw))
                        wrong.extend((s, n) for a, b in zip(got, want[s][n]) if not torch.equal(a, b))
        except Exception as e:      # noqa: BLE001 -- said by the test's own thread
            wrong.append((s, e))
    threads = [threading.Thread(target=run, args=(s,)) for s in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
