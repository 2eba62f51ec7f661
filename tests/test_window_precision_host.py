"""What window attention's header says of q, by arithmetic on the CPU: values split into e4m3
parts as the kernel for head_dim 128 splits them."""
import pytest
import torch

from tests.window_ref import e4m3


@pytest.mark.parametrize("dtype,parts,exact", [(torch.bfloat16, 2, -9), (torch.float16, 3, -6)])
def test_q_in_parts(dtype, parts, exact):
    # the row's largest magnitude is scaled into [2^7, 2^8); every value below it, in each binade
    bits = 8 if dtype == torch.bfloat16 else 11
    grid = torch.arange(2 ** (bits - 1), 2 ** bits, dtype=torch.float64) * 2.0 ** (1 - bits)
    for binade in range(-30, 1):
        x = grid * 2.0 ** (7 + binade)
        rest = x.clone()
        for _ in range(parts):
            rest -= e4m3(rest)
        assert rest.abs().max() <= 2.0 ** (7 - 17)
        assert (rest == 0).all() == (binade >= exact)


def e5m2(x):
    return x.to(torch.float8_e5m2).double()


def every_probability():
    """fp16 values from 0 to 2^8."""
    return torch.arange(0, 0x5C01, dtype=torch.int16).view(torch.float16).double()


def test_p_in_three_parts_of_e4m3():
    p = every_probability()
    c0 = e4m3(p)
    c1 = e4m3((p - c0) * 2.0 ** 5)
    c2 = e4m3(((p - c0) * 2.0 ** 5 - c1) * 2.0 ** 5)
    off = (c0 + c1 * 2.0 ** -5 + c2 * 2.0 ** -10 - p).abs()
    assert off.max() <= 2.0 ** -20 and (off[p >= 2.0 ** -9] == 0).all()


def test_p_in_two_types():
    p = every_probability()
    c0 = e4m3(p)
    c1 = e5m2(p - c0)
    c2 = e4m3((p - c0 - c1) * 2.0 ** 9)
    off = (c0 + c1 + c2 * 2.0 ** -9 - p).abs()
    assert off.max() <= 2.0 ** -19 and (off[p >= 2.0 ** -8] == 0).all()
