"""The split of P that the e4m3 kernel makes for chosen blocks, over all of its
range: hi rounded to 4 significant bits, lo what that leaves, both e4m3.
"""
import torch


def _e4m3(x):
    return x.to(torch.float8_e4m3fn).float()


def _split(p16):
    """As the kernel does: half a step of the leading bits added to the fp16 pattern, then cut."""
    bits = p16.view(torch.int16).int() & 0xFFFF
    hi = ((bits + 0x40) & 0xFF80).to(torch.int16).view(torch.float16)
    rest = p16.float() - hi.float()
    assert torch.equal(rest.half().float(), rest)               # exact in fp16
    return _e4m3(hi.float()), _e4m3(rest), hi.float()


def test_rounded_split_bound_over_every_fp16_up_to_448():
    p16 = torch.arange(0, 0x5F01, dtype=torch.int32).to(torch.int16).view(torch.float16)
    p = p16.float()
    assert p[-1] == 448.0 and (28.0 * 8 * 2) == 448.0           # norm, lazy maximum, scale slack
    hi, lo, exact = _split(p16)
    assert bool((exact <= 448.0).all()) and bool((hi >= 0).all())
    normal = exact >= 2.0 ** -6
    assert torch.equal(hi[normal], exact[normal])
    err = (p - hi - lo).abs()
    # lo is at most half a step of hi's four bits, 2^-4 of hi's leading bit, and keeps four of its own: half a step
    # 2^-5 of its leading bit, or half of e4m3's smallest step 2^-9.  Below 2^-6 hi meets that step too.
    bound = torch.maximum(2.0 ** -9 * p, torch.full_like(p, 2.0 ** -10))
    assert bool((err <= bound)[p >= 2.0 ** -6].all())
    assert bool((err <= 2.0 ** -9)[p < 2.0 ** -6].all())


def test_negative_values_split_as_their_magnitude():
    p16 = torch.arange(0, 0x5F01, dtype=torch.int32).to(torch.int16).view(torch.float16)
    (a, b, _), (c, d, _) = _split(p16), _split(-p16)
    assert torch.equal(a, -c) and torch.equal(b, -d)
