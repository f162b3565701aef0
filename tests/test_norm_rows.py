"""Refusals of the layer normalisation's rows that are one (no GPU: the addresses must not be read)."""
import struct

import onnx_recurrent_gb300 as orc

AT, FAR = 4096, 1 << 30


def test_rows_that_are_one_are_an_inputs():
    orc.build()
    from onnx_recurrent_gb300 import norm
    lib = norm._load()
    p = orc.rnn_norm_create(16)
    for fields, text in ([3, AT, 0, 0, 0, FAR, -1, 0, 0], "Y has a negative stride"), ([3, AT, -2, 0, 0, FAR, 0, 0, 0], "X has a negative stride"), \
            ([3, AT, -1, 0, 0, AT, 0, 0, 0], "X and Y overlap in part"):
        assert lib.rnn_layer_norm(p.handle, struct.pack("9q", *fields)) == 1
        assert text in orc.rnn_last_error()
