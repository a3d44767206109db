"""Int4Experts and decode_i4 refuse codes and scales that do not belong to the layer or to the group."""
import pytest
import torch

import mixture_experts_layer_02_amd as moe

NL, D, F = 4, 256, 128


def _parts(group, device="cpu", n=NL, d=D, f=F):
    out = []
    for rows, cols in ((f, d), (f, d), (d, f)):
        out += [torch.full((n, rows, cols // 2), 0x88, dtype=torch.uint8, device=device),
                torch.ones(n, rows, -(-cols // group), device=device)]
    return out


@pytest.mark.parametrize("group", [0, 16, -128, 256])
def test_groups_are_checked_when_experts_are_made(group):
    w = torch.zeros(2, 8, 64)
    with pytest.raises(ValueError):
        moe.Int4Experts(w, w, w, group=group)
    with pytest.raises(ValueError):
        moe.Int4Experts.from_codes(*_parts(32), group=group)


@pytest.mark.parametrize("made,named", [(32, 128), (64, 128), (32, 64), (128, 32), (64, 32)])
def test_scales_of_another_group_are_refused(made, named):
    with pytest.raises(ValueError, match="w1s"):
        moe.Int4Experts.from_codes(*_parts(made), group=named)
    parts = _parts(named)
    parts[5] = _parts(made)[5]
    with pytest.raises(ValueError, match="w2s"):
        moe.Int4Experts.from_codes(*parts, group=named)
    moe.Int4Experts.from_codes(*_parts(made), group=made)


@pytest.mark.gpu
def test_decode_refuses_experts_of_another_layer(gpu):
    b = moe.DecodeBuffers(moe.make_desc(3, D, F, 8, 2, 4, NL, "bf16"))
    x, wr = torch.ones(3, D, dtype=torch.bfloat16, device=gpu), torch.ones(8, D, dtype=torch.bfloat16, device=gpu)

    def step(parts, group=64):
        return moe.decode_i4(b, x, wr, moe.Int4Experts.from_codes(*parts, group=group))

    ok = _parts(64, gpu)
    assert (step(ok) == 0).all()
    assert (step([t.flatten() for t in ok]) == 0).all()      # laid out the same, told by their number
    assert (step([t.flatten(0, 1) for t in ok]) == 0).all()
    assert (step(_parts(64, gpu, n=NL + 2)) == 0).all()      # the first NL of more experts
    for bad in (_parts(64, gpu, n=NL - 1), _parts(64, gpu, d=2 * D), _parts(64, gpu, f=2 * F), _parts(64, gpu, d=F, f=D),
                [t.flatten() for t in _parts(64, gpu, n=NL + 2)], ok[:1] + [_parts(32, gpu)[1].flatten()] + ok[2:],
                ok[:5] + [_parts(32, gpu)[5].flatten(0, 1)]):
        with pytest.raises(ValueError):
            step(bad)
    e = moe.Int4Experts.from_codes(*_parts(32, gpu), group=32)
    e.group = 64  # (set afterwards)
    with pytest.raises(ValueError):
        moe.decode_i4(b, x, wr, e)
