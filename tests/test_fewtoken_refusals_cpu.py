"""Tensors that are not on a GPU are refused with ValueError, also where there is no GPU at all."""
import pytest

import w4a4_quantized_linear_amd as sq

torch = pytest.importorskip("torch")


def test_host_tensors():
    layer, down = sq.Layer("mxfp4", 512, 1024, 0), sq.Layer("mxfp4", 512, 32, 0)
    X = torch.zeros((2, 512), dtype=torch.bfloat16)
    w, wd = (torch.zeros((1, sq.weight_bytes(l)), dtype=torch.uint8) for l in (layer, down))
    ids, wt = torch.zeros((2, 1), dtype=torch.int32), torch.zeros((2, 1))
    for call in (lambda: sq.linear_w4a16(layer, w[0], X), lambda: sq.moe_route(X, X, 1),
                 lambda: sq.moe(layer, w, down, wd, X, ids, wt), lambda: sq.pack_experts(layer, torch.zeros((1, 1024, 512)))):
        with pytest.raises(ValueError):
            call()
