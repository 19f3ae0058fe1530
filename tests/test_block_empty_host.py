"""The gradient of a block whose output has no rows, without a GPU: the C entry takes
no address for a buffer of no rows, where slots say that there is one."""
import ctypes

import top_routing_expert_gb300 as moe


def test_no_rows_and_no_output():
    moe.build()
    lib = moe.load_library()
    f, off = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)  # never dereferenced

    def bwd(rows, y, dest, ws):
        b = moe._Block(4, 128, rows, 2, 1, 1.0, 1e-6)
        return lib.moe_block_norm_bwd(ctypes.byref(b), f, y, dest, f, f, f, f, f, f, f, None, f, f,
                                      f, f, ws, 1 << 30, None)

    # accepted as far as the workspace, the last of the checks
    assert bwd(0, None, f, off) == 5 and bwd(0, None, f, None) == 1
    assert bwd(8, None, f, off) == 1       # rows without an address
    assert bwd(0, None, None, off) == 1    # no block output: gradients of what is not there
