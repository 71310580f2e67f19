"""A stream on a part of the device's SMs (a green context), by the driver's own interface."""
import contextlib
import ctypes

_RES = ctypes.c_uint32 * 256      # room for a CUdevResource; the SMs' count follows its type and padding, at byte 96
_SM, _DEFAULT_STREAM, _NON_BLOCKING = 1, 1, 1


def sm_count(resource):
    return resource[96 // 4]


@contextlib.contextmanager
def stream_on_part(min_sms):
    """(driver library, stream handle, its SMs): a stream of a green context of at least `min_sms` SMs."""
    cu = ctypes.CDLL("libcuda.so.1")

    def ok(rc):
        assert rc == 0, rc

    dev, whole, part, rest, n = ctypes.c_int(), _RES(), _RES(), _RES(), ctypes.c_uint(1)
    ok(cu.cuDeviceGet(ctypes.byref(dev), 0))
    ok(cu.cuDeviceGetDevResource(dev, whole, _SM))
    ok(cu.cuDevSmResourceSplitByCount(part, ctypes.byref(n), whole, rest, 0, min_sms))
    desc, green, stream = (ctypes.c_void_p() for _ in range(3))
    ok(cu.cuDevResourceGenerateDesc(ctypes.byref(desc), part, 1))
    ok(cu.cuGreenCtxCreate(ctypes.byref(green), desc, dev, _DEFAULT_STREAM))
    try:
        ok(cu.cuGreenCtxStreamCreate(ctypes.byref(stream), green, _NON_BLOCKING, 0))
        got = _RES()
        ok(cu.cuGreenCtxGetDevResource(green, got, _SM))
        yield cu, stream, sm_count(got)
        ok(cu.cuStreamSynchronize(stream))
        ok(cu.cuStreamDestroy_v2(stream))
    finally:
        ok(cu.cuGreenCtxDestroy(green))
