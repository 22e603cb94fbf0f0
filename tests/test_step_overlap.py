"""Refusals of the step operators where an output's memory meets something else (include/bitdelta_step.h says what has
to lie apart): the binding's checks, on host tensors."""

import pytest
import torch

import tenant_serving_amd as bd

BF, E4 = torch.bfloat16, torch.float8_e4m3fn


def test_scales_apart_from_each_other_and_from_the_codes():
    k, v = (torch.zeros((6, 2, 16, 64), dtype=torch.uint8).view(E4) for _ in range(2))
    n = 6 * 2 * 16
    s = torch.zeros(3 * n, dtype=torch.uint8)
    one = s[:n].view(6, 2, 16)
    for a, b, match in ((one, one, "k_scales overlaps v_scales"),
                        (one, s[n - 8:2 * n - 8].view(6, 2, 16), "k_scales overlaps v_scales"),
                        (s[n - 8:2 * n - 8].view(6, 2, 16), one, "k_scales overlaps v_scales"),
                        (k.view(torch.uint8).view(-1)[128:128 + n].view(6, 2, 16), one, "k_scales overlaps k"),
                        (one, v.view(torch.uint8).view(-1)[-n:].view(6, 2, 16), "v_scales overlaps v"),
                        (one, k.view(torch.uint8).view(-1)[:n].view(6, 2, 16), "v_scales overlaps k"),
                        (one, s[n:2 * n].view(6, 2, 16), "GPU")):
        with pytest.raises(ValueError, match=match):
            bd.bd_kv_cache(k, v, a, b)
    # one allocation of pages with room behind each row's codes: the scales may lie between rows, not on them
    wide = torch.zeros((2, 2, 16, 256), dtype=torch.uint8)
    k, v = wide[:1, :, :, :64].view(E4), wide[1:, :, :, :64].view(E4)
    row = wide[0, 0, 0]
    with pytest.raises(ValueError, match="GPU"):
        bd.bd_kv_cache(k, v, row[64:96].view(1, 2, 16), row[96:128].view(1, 2, 16))
    with pytest.raises(ValueError, match="k_scales overlaps k"):
        bd.bd_kv_cache(k, v, row[56:88].view(1, 2, 16), row[96:128].view(1, 2, 16))
    with pytest.raises(ValueError, match="v_scales overlaps k"):
        bd.bd_kv_cache(k, v, row[64:96].view(1, 2, 16), row[232:].as_strided((1, 2, 16), (32, 16, 1)))
