"""What the parts of 8 bits that attention over an 8-bit cache splits its operands into leave of them, over all values of the types:
the errors that ar.h states."""
import pytest
import torch

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def to(x, t):
    return x.float().to(t).double()


def elements(dt):
    """Every magnitude that an element of a row has when the row's largest is brought to 224 .. 448, down to where its parts are zeros."""
    x = torch.arange(1 << 15, dtype=torch.int32).to(torch.int16).view(dt)
    x = x[torch.isfinite(x)].double()
    x = torch.unique(torch.cat([x * 2.0 ** e for e in range(-25, 26)]))
    return x[(x > 2.0 ** -30) & (x <= 448.0)]


@pytest.mark.parametrize("dt, parts, exact_from", [(torch.bfloat16, 2, 2.0 ** -6), (torch.float16, 3, 2.0 ** -3)])
def test_query_parts(dt, parts, exact_from):
    """E4M3, E4M3 again in fp16, the rest in E5M2."""
    x = elements(dt)
    rest = x.clone()
    for _ in range(parts - 1):
        rest = rest - to(rest, E4M3)
    rest = (rest - to(rest, E5M2)).abs()
    assert (rest[x >= exact_from] == 0).all()
    assert rest.max() == 2.0 ** -14  # 2^-21.8 of 224


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_query_parts_for_few_rows(dt):
    """Three E4M3 parts, each of the rest of the one before times 16."""
    rest, unit = elements(dt), 1.0
    for i in range(3):
        assert rest.max() <= 448.0
        rest = rest - to(rest, E4M3)
        if i < 2:
            rest, unit = rest * 16.0, unit / 16.0
    assert (rest.abs() * unit).max() == 2.0 ** -18  # 2^-25.8 of 224
