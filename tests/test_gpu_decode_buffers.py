"""One set of DecodeBuffers, made for the most tokens, serves steps of fewer."""
import pytest
import torch

import mixture_experts_layer_02_amd as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [0, 64])
def test_steps_of_fewer_tokens_in_the_same_buffers(gpu, group):
    d, f, E, k = 512, 256, 32, 4
    g = torch.Generator(device="cuda").manual_seed(3)

    def rand(std, *shape):
        return torch.empty(shape, dtype=torch.bfloat16, device=gpu).normal_(0, std, generator=g)

    w = rand(0.05, E, f, d), rand(0.05, E, f, d), rand(0.05, E, d, f)
    wr, bias = rand(d ** -0.5, E, d), torch.randn(E, generator=g, device=gpu)
    experts = moe.Int4Experts(*w, group=group) if group else None

    def step(b, x):
        if group:
            return moe.decode_i4(b, x, wr, experts, bias=bias)
        return moe.decode(b, x, wr, *w, bias=bias)

    def desc(T):
        return moe.make_desc(T, d, f, E, k, 0, E, "bf16")

    most = moe.DecodeBuffers(desc(64))
    for T in (64, 1, 17, 2, 63, 9, 64, 5):
        x = rand(1.0, T, d)
        own = moe.DecodeBuffers(desc(T))
        step(own, x)
        most.desc = desc(T)
        for t in (most.y, most.topk_idx, most.topk_w):
            t.fill_(77)
        assert step(most, x) is most.y
        for name in ("y", "topk_idx", "topk_w"):
            got = getattr(most, name)
            assert torch.equal(got[:T], getattr(own, name)) and (got[T:] == 77).all(), (T, name)
    with pytest.raises(ValueError):  # more tokens than the buffers have room for
        small = moe.DecodeBuffers(desc(4))
        small.desc = desc(5)
        step(small, rand(1.0, 5, d))
