"""First calls of the int8 binding from several threads, without a GPU."""

import threading

import w4a16_group_quantized_qmv_amd as w4
from w4a16_group_quantized_qmv_amd import mxfp4, w8a8

from test_w8a8_cpu import PYTHON, arguments, model  # noqa: F401  (model is a fixture)


class Watched:
    """Passes lookups on and calls ``seen`` before each."""

    def __init__(self, inner, seen):
        self.__dict__.update(inner=inner, seen=seen)

    def __getattr__(self, name):
        self.seen()
        return getattr(self.inner, name)


def test_a_first_call_beside_another_thread_s(model, monkeypatch):  # noqa: F811
    """Another thread's first call comes before the n-th lookup of this one's, for every n: it goes through, with
    outputs of the right types."""
    torch, recorder = model
    a = arguments(torch)
    results, lookups, at = [], 0, 0

    def run():
        try:
            codes, scales = PYTHON["w8a8_quantize_rows"](a, {})
            results.append((codes.dtype, scales.dtype))
        except Exception as error:                           # noqa: BLE001  (what the other thread saw)
            results.append(error)

    def seen():
        nonlocal lookups
        if threading.current_thread() is not threading.main_thread():
            return
        lookups += 1
        if lookups == at:
            t = threading.Thread(target=run)
            t.start()
            t.join()

    watched = Watched(torch, seen), Watched(recorder, seen)
    for module in (w4, mxfp4, w8a8):
        monkeypatch.setattr(module, "_torch", lambda: watched[0])
    monkeypatch.setattr(w8a8, "load", lambda: watched[1])
    while lookups == at:                                     # (until a call has fewer than n)
        lookups, at = 0, at + 1
        w8a8._FN = {}
        w8a8._BF16 = w8a8._FP32 = w8a8._I8 = w8a8._I32 = mxfp4._T = None
        PYTHON["w8a8_linear"](a, {})
        lookups = min(lookups, at)
    assert at > 15 and len(results) == at - 1 and set(results) == {("int8", "float32")}, results
