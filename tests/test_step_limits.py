"""The largest sizes that include/bitdelta_step.h names, on the host: one step past each is refused before anything is
enqueued, and the workspace query has no answer for it."""

import ctypes

from tenant_serving_amd import step

FAKE = 1 << 20          # 16-byte aligned, never dereferenced
OK, SHAPE, WORKSPACE = 0, 2, 4


def _attend(lib, B, heads, group, page, pages):
    """The call's answer with no workspace, which a call within the limits that splits its rows asks for first."""
    kv = step._KV(k=FAKE, v=FAKE, type=0, num_heads=heads, head_dim=64, page_size=page, num_pages=10,
                  page_stride=heads * page * 64, head_stride=page * 64, token_stride=64)
    pair = step._Pair(heads * group * 64, 64)
    return lib.bd_attend(ctypes.byref(kv), FAKE, 0, pair, heads * group, FAKE, pages, pages, FAKE, B, 0.1, FAKE, None,
                         None, 0, None)


def test_attention_limits():
    lib = step._library()
    for fine, past in (((1, 1, 1, 16, 1 << 20), (1, 1, 1, 16, (1 << 20) + 1)),             # 2^24 tokens of a sequence
                       ((1 << 18, 8, 4, 16, 4064), (1 << 18, 8, 4, 16, 4065)),             # R * (U + 4) = 2^21 * 512
                       ((1 << 16, 8, 17, 16, 8160), (1 << 16, 8, 17, 16, 8161)),           # two tiles of query heads
                       ((1 << 20, 8, 1, 128, 100), ((1 << 20) + 1, 8, 1, 128, 100))):      # R = 2^23
        assert lib.bd_attend_workspace_bytes(fine[0], fine[1] * fine[2], fine[1], 64, *fine[3:]) > 0, fine
        assert _attend(lib, *fine) == WORKSPACE, fine
        assert lib.bd_attend_workspace_bytes(past[0], past[1] * past[2], past[1], 64, *past[3:]) == 0, past
        assert _attend(lib, *past) == SHAPE, past


def test_token_limits():
    lib = step._library()
    kv = step._KV(k=FAKE, v=FAKE, type=0, num_heads=2, head_dim=64, page_size=16, num_pages=10, page_stride=2048,
                  head_stride=1024, token_stride=64)
    pair = step._Pair(128, 64)
    assert lib.bd_kv_write(ctypes.byref(kv), FAKE, pair, FAKE, pair, 0, FAKE, (1 << 28) + 1, None) == SHAPE
    assert lib.bd_kv_read(ctypes.byref(kv), FAKE, 1 << 31, FAKE, FAKE, None) == SHAPE
    assert lib.bd_rms_norm(FAKE, 0, None, None, 0, FAKE, 0, 1, None, 1e-5, FAKE, 0, None, 1 << 31, 64, None) == SHAPE
