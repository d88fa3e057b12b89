"""grad_norm's refusals of buffers that overlap, which come before any CUDA call."""
import ctypes


from test_abi_host import A, BF16, EOVERLAP, F32
from test_many_host import B, C, D, lib  # noqa: F401  (the fixture)


def test_the_norm_and_the_workspace_overlap_nothing(lib):  # noqa: F811
    def call(norm=C, ws=D, numels=(100, 7)):
        return lib.grad_norm((ctypes.c_void_p * 2)(A, B), (ctypes.c_int64 * 2)(*numels), (ctypes.c_int * 2)(F32, BF16),
                             2, norm, ws, 1 << 20, None)

    for norm in (A, A + 396, B, B + 12, D, D + 64):
        assert call(norm=norm) == EOVERLAP
    for ws in (A, A + 392, A - 64, B + 8, C):
        assert call(ws=ws) == EOVERLAP
