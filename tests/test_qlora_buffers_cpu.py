"""The buffers that a captured step keeps."""

import torch

from bit_grouped_moe_e4b_b200 import qlora


def test_a_buffer_stays_where_it_is():
    buf = qlora.Buffers()
    one = buf("h", (4, 8), torch.float32, "cpu")
    at = one.data_ptr()
    del one
    kinds = [((5, 8), torch.float32), ((4, 8), torch.bfloat16), ((32,), torch.float32), ((4, 8), torch.float32)]
    others = [buf("h", shape, dtype, torch.device("cpu")) for shape, dtype in kinds]
    assert [o.shape for o in others] == [torch.Size(s) for s, _ in kinds] and [o.dtype for o in others] == [d for _, d in kinds]
    # the first is still held, and comes again for its shape and type
    assert others[-1].data_ptr() == at and len({o.data_ptr() for o in others}) == 4
    assert buf("x", (4, 8), torch.float32, "cpu").data_ptr() != at
