"""The append of many tokens, whose CTAs take several vectors a lane at a time: every layout, type and pairing against the
64-bit oracle (needs a GB300)."""
import pytest

from test_gpu_kv_append import Q, Step  # noqa: F401 (Q is a fixture)

pytestmark = pytest.mark.gpu

# a CTA's 128 threads hold 8 vectors of 128 or 16 of 64 at a time; four query vectors a lane (up to 32 or 64 query heads) or
# eight, numbers of heads that are no multiples of these, more cached vectors than query heads, no query heads
LAYOUTS = [(64, 8, 128, 128, False), (128, 64, 128, 64, True), (33, 11, 128, 24, True), (100, 4, 128, 96, False),
           (9, 3, 128, 0, False), (0, 12, 128, 128, True), (7, 7, 64, 24, True), (20, 5, 64, 64, False), (0, 16, 64, 32, False),
           (70, 7, 64, 32, True), (65, 13, 64, 64, False)]


@pytest.mark.parametrize("hq,hkv,dim,rotary,interleaved", LAYOUTS)
@pytest.mark.parametrize("e2m1,f16,norm,factors", [(True, False, True, (1.0, 1.0)), (False, True, False, (0.3, 5.0)),
                                                   (False, False, True, (0.25, 2.0 ** -7)), (True, True, False, (1.0, 3.0))])
def test_many_tokens(Q, hq, hkv, dim, rotary, interleaved, e2m1, f16, norm, factors):  # noqa: F811
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    # (more than 16 CTAs an SM when a group of lanes has one vector)
    slices = -(-(hq + 2 * hkv) // (1024 // dim))
    assert slices > 1
    s = Step(16 * sms // slices + 3, hq, hkv, dim, rotary, e2m1, f16, interleaved, norm, factors, seed=hq + rotary, block_size=64)
    s.check(s.run(Q, packed=interleaved, in_place=norm))
