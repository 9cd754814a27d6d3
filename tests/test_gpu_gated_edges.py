"""The gated block's calls at their edges: rows that are alike, and values at
the ends of the range."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def gq():
    import __graft_entry__

    __graft_entry__.build()
    import fp8_quantization_moe_gb300 as m

    return m


def blocks(n):
    return -(-n // 128)


def codes(gen, *shape):
    return (100 * torch.randn(*shape, device=DEV, generator=gen)).clamp(-448, 448).to(E4M3)


def scales(gen, *shape):
    return 300 + 300 * torch.rand(*shape, device=DEV, generator=gen)


# M, inner, outer, offs: few tiles, whose contraction two, four (and for few rows eight)
# blocks share, and many, that one block or a pair takes
ALIKE = [
    (16, 2064, 272, [16]), (23, 4112, 128, [3, 23]), (128, 2704, 272, [128]), (140, 7184, 768, [9, 140]),
    (300, 2704, 1040, [1, 300]), (700, 2800, 528, [257, 300, 300, 700]), (6200, 144, 2576, [3000, 3001, 6200]),
    (2000, 1024, 512, [130, 2000]),
]


def same_rows(t, offs):
    flat = t.flatten(1).view(torch.uint8)
    start = 0
    for end in offs:
        if end > start:
            assert torch.equal(flat[start:end], flat[start:start + 1].expand(end - start, -1))
        start = end


@pytest.mark.parametrize("M,inner,outer,offs", ALIKE)
def test_rows_that_are_alike(gq, M, inner, outer, offs):
    """Equal rows of a group get equal bits, wherever in their tile they are."""
    gen = torch.Generator(device=DEV).manual_seed(M)
    E = len(offs)
    ends = torch.tensor(offs, dtype=torch.int32, device=DEV)
    qa = codes(gen, 1, inner).view(torch.uint8).expand(M, -1).contiguous().view(E4M3)
    sa = scales(gen, 1, blocks(inner)).expand(M, -1).contiguous()
    qb, sb = codes(gen, E, 2, outer, inner), scales(gen, E, 2, blocks(outer), blocks(inner))
    r = gq.grouped_gated_mm(qa, sa, qb, sb, ends, fp8=True, keep=True)
    gq.check_device_error()
    for t in r:
        same_rows(t, offs)
    qd = codes(gen, 1, 2, inner).view(torch.uint8).expand(M, -1, -1).contiguous().view(E4M3)
    sd = scales(gen, 1, 2, blocks(inner)).expand(M, -1, -1).contiguous()
    qb, sb = codes(gen, E, 2, inner, outer), scales(gen, E, 2, blocks(inner), blocks(outer))
    out = gq.grouped_gated_grad(qd, sd, qb, sb, ends)
    gq.check_device_error()
    same_rows(out, offs)
