"""Pins of the plain implementations that the step operators' GPU tests compare with: the e4m3 table against torch's
own conversions on the host, the attention and the norm against torch in 64 bits."""

import numpy as np
import torch

from tests import step_reference as ref


def test_the_table_is_the_format():
    codes = torch.arange(256, dtype=torch.uint8)
    ours = ref.decode(codes.numpy(), 127)
    theirs = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(ours), np.isnan(theirs))
    assert np.array_equal(ours[~np.isnan(ours)], theirs[~np.isnan(theirs)])


def test_encoding_agrees_with_torch():
    gen = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(20000, generator=gen) * 100, torch.randn(20000, generator=gen) * 2.0 ** -7,
                   torch.from_numpy((ref.E4M3[1:] + ref.E4M3[:-1]) / 2).float(), -torch.from_numpy(ref.E4M3).float()])
    x = x.clamp(-448, 448)
    assert np.array_equal(ref.encode(x.double().numpy(), 127), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_scale_byte_is_the_smallest():
    for a in (0.0, 1e-40, 448 * 2.0 ** -111, 449 * 2.0 ** -111, 1.0, 1.75, 1.7500001, 448.0, 448.001, 3.3e38):
        b = ref.scale_byte(a)
        assert a <= 448 * 2.0 ** (b - 127) and b >= 16
        assert b == 16 or a > 448 * 2.0 ** (b - 128)
    assert ref.scale_byte(1.75) == 127 - 8 and ref.scale_byte(1.75 * (1 + 2 ** -23)) == 127 - 7


def test_attention_and_norm_agree_with_torch():
    gen = torch.Generator().manual_seed(2)
    q = torch.randn((6, 32), generator=gen, dtype=torch.float64)
    k, v = (torch.randn((19, 2, 32), generator=gen, dtype=torch.float64) for _ in range(2))
    out, lse, _ = ref.attend(q.numpy(), k.numpy(), v.numpy(), 0.25)
    kk, vv = (t.permute(1, 0, 2).repeat_interleave(3, 0) for t in (k, v))
    s = (kk @ q[:, :, None])[..., 0] * 0.25
    want = (torch.softmax(s, 1)[:, None, :] @ vv)[:, 0]
    assert np.allclose(out, want.numpy(), rtol=1e-12, atol=1e-14)
    assert np.allclose(lse, torch.logsumexp(s, 1).numpy(), rtol=1e-12)
    x = torch.randn((3, 40), generator=gen)
    g = torch.randn((1, 40), generator=gen)
    y, _ = ref.rms_norm(x, g, 1e-5)
    assert np.allclose(y, torch.nn.functional.rms_norm(x.double(), (40,), g[0].double(), 1e-5).numpy(), rtol=1e-12)
