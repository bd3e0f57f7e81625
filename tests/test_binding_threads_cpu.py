"""The binding looks torch up at its first call, which several threads may make."""
import sys

from bit_expert_ffn_fp32_b200 import native


def test_what_callers_look_at_is_there_last():
    """At every line of the look-up: where `device` or `code` is set, all that a call
    then uses is set as well."""
    T = native._Types
    T.code, T.int32, T.device, T.raw_stream = {}, None, None, None
    seen = []

    def trace(frame, event, arg):
        if frame.f_code is T.load.__func__.__code__:
            ready = T.int32 is not None and T.raw_stream is not None
            seen.append(ready or (T.device is None and not T.code))
            return trace
        return None

    sys.settrace(trace)
    try:
        T.load()
    finally:
        sys.settrace(None)
        complete = bool(T.code) and None not in (T.int32, T.device, T.raw_stream)
        T.code, T.int32, T.device, T.raw_stream = {}, None, None, None
        T.load()
    assert complete and len(seen) > 5 and all(seen)
