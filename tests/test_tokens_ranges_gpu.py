"""The operators around the experts at the far ends of what they are given."""
import numpy as np
import pytest

import moe_expert_token_gb300 as moe
import moe_expert_token_gb300.mrr_v2 as m
from oracle import tokens as ox
from test_experts_gpu import down, up
from test_tokens_together_gpu import example

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from moe_expert_token_gb300 import build

    build.build()
    m.load_library()


@pytest.mark.parametrize("quant", ["int8", "e4m3", "e4m3_128"])
@pytest.mark.parametrize("exponent", [-126, -122, -119, -116, -112, -105, -98, -65, -56, 0, 100])
def test_codes_of_quotients_at_ties(quant, exponent):
    """Elements as near as float32 comes to the middle between two codes, under scales from 2^-126 up: each code is that of y / s
    in float32, to the bit.  Rows below 2^-20 under an eps of 1 have r = 1, and weights of a power of two give any y."""
    T, H = 200, 1024
    rng = np.random.default_rng(exponent + 200)
    block, top = (128 if quant == "e4m3_128" else H), np.float32(127 if quant == "int8" else 448)
    values = np.arange(128.0) if quant == "int8" else ox.E4M3
    largest = np.ldexp((1 + rng.integers(0, 2 ** 23, (T, H // block)) * 2.0 ** -23).astype(np.float32), exponent)
    s = np.maximum(largest / top, np.float32(2.0 ** -126))
    each, most = np.repeat(s, block, axis=1), np.repeat(largest, block, axis=1)
    i = rng.integers(0, len(values) - 1, (T, H))
    tie = ((values[i] + values[i + 1]) / 2 * each.astype(np.float64)).astype(np.float32)
    y = np.minimum(tie, most) * rng.choice([-1, 1], (T, H)).astype(np.float32)
    y[:, ::block] = largest
    x = np.ldexp(y, -exponent - 20)
    w = np.full(H, 2.0 ** (exponent + 20), np.float32)
    got, _, q, scales = moe.moe_add_rms_norm(up(x, "float32"), up(w, "float32"), eps=1.0, quant=quant)
    assert np.array_equal(down(got), y.astype(np.float64))
    assert np.array_equal(down(scales).reshape(s.shape), s.astype(np.float64))
    v = y / each
    want = np.clip(np.rint(v), -127, 127) if quant == "int8" else ox.nearest(v.astype(np.float64), ox.E4M3)
    assert np.array_equal(down(q.float()), want)


def test_block_of_many_ranks():
    """More (rank, expert) pairs than one sort takes (4096): the block's result is the one that few ranks give.  A row's products
    do not depend on where it lies, so the results are equal to the bit.  Token t chooses experts k t .. k t + k - 1 (mod E), which
    its logits say by themselves, so every pair has rows."""
    import torch

    block = example("moe_block")
    gen = torch.Generator(device="cuda").manual_seed(1)
    T, E, I, k = 16384, 128, 64, 8
    w = block.weights(E, E, I, gen) | {"router": torch.eye(E, device="cuda").bfloat16(), "bias": torch.zeros(E, device="cuda").bfloat16()}
    expert = (k * torch.arange(T, device="cuda")[:, None] + torch.arange(k, device="cuda")) % E
    x = (0.125 * torch.randn(T, E, generator=gen, device="cuda")).scatter_add_(1, expert, torch.full((T, k), 6.0, device="cuda")).bfloat16()
    few = block.prefill(x, w, k, ranks=2)
    for ranks in (32, 33, 40):                  # 4096 pairs, and more of them in shares of equal and of different sizes
        assert torch.equal(block.prefill(x, w, k, ranks=ranks), few)


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
@pytest.mark.parametrize("norm_type", [0, 1, 2])
def test_training_example_routes_with_biases(dt, norm_type):
    """GatingTopK with a bias, and with a second one for the rows of a mask: the gradients that float64 gives the same weights,
    within the kernel's bound for them (as tests/test_tokens_gpu.py holds it)."""
    import torch

    from test_tokens_gpu import close

    block = example("moe_training")
    T, e, k = 50, 24, 4
    rng = np.random.default_rng(norm_type)
    logits, bias, extra = up(2 * rng.standard_normal((T, e)), dt), up(0.3 * rng.random(e), dt), up(0.5 * rng.random(e), dt)
    gy, mask = up(rng.standard_normal((T, k)), dt), up(rng.random(T) < 0.5)
    routing = dict(norm_type=norm_type, routed_scaling_factor=2.5)
    for second in (None, extra):
        leaves = [t.clone().requires_grad_() for t in (logits, bias) + (() if second is None else (second,))]
        more = {} if second is None else {"additional_token_mask": mask}
        weight, expert = block.GatingTopK.apply(leaves[0], k, routing | more, *leaves[1:])
        weight.backward(gy)
        ref = ox.gating_grad(down(gy), down(logits), expert.cpu().numpy(), bias=down(bias), scale=2.5, norm_type=norm_type,
                             additional_bias=None if second is None else down(second),
                             mask=None if second is None else mask.cpu().numpy())
        ops = 3 * (e / 32 + k / 32) + 120
        for leaf, i in zip(leaves, (0, 2, 4)):
            close(leaf.grad, ref[i], ref[i + 1], ops + (T / 64 + 60 if i else 0), dt)
    with pytest.raises(TypeError):              # a bias among the plain settings would get no gradient
        block.GatingTopK.apply(logits, k, routing | {"bias": bias}, bias)


@pytest.mark.parametrize("T,k,held", [(1, 8, 16), (300, 3, 16), (300, 3, 5), (9000, 8, 2)])
def test_gradient_of_the_sorted_weights(T, k, held):
    """Each slot's weight has the gradient of its row's, and 0 without a row: a combine with one slot a token."""
    import torch

    rng = np.random.default_rng(T)
    idx = torch.from_numpy(rng.integers(0, 16, (T, k))).int().cuda()
    x, weight = torch.ones((T, 4), device="cuda"), torch.rand((T, k), device="cuda")
    _, _, _, row_idx, _, moved = moe.moe_sort_tokens(x, idx, held, expert_topk_weight=weight)
    grad = torch.randn(moved.shape, device="cuda")
    got = moe.moe_combine_tokens(grad, row_idx.view(-1, 1)).view(T, k)
    want = torch.where(row_idx >= 0, grad[row_idx.clamp(min=0).long(), 0], torch.zeros((), device="cuda"))
    assert torch.equal(got, want)
