"""The operators around the experts together, as the examples use them."""
import importlib.util
import os

import numpy as np
import pytest

import moe_expert_token_gb300 as moe
import moe_expert_token_gb300.mrr_v2 as m
from oracle import experts as oe
from oracle import tokens as ox
from test_experts_gpu import down

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from moe_expert_token_gb300 import build

    build.build()
    m.load_library()


def example(name):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", name + ".py")
    spec = importlib.util.spec_from_file_location(name, path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_block_with_its_norm_in_front():
    """examples/moe_block.py: residual, norm and MXFP4 rows, tokens sorted, re-routed, through the experts and back,
    against the same steps in the oracle, given the GPU's own routing.  The norm's float32 y moves a code of the rows as
    rarely as 2^-20; each expert's result is rounded to bfloat16 (2^-9 of it, 2^-10 root mean square) and the sum once
    more: the whole within 2^-8."""
    import torch

    block = example("moe_block")
    gen = torch.Generator(device="cuda").manual_seed(3)
    T, E, H, I, k = 256, 8, 256, 128, 4
    w = block.weights(E, H, I, gen)
    x, res = (torch.randn(T, H, generator=gen, device="cuda").bfloat16() for _ in range(2))
    gain = (1 + 0.1 * torch.randn(H, generator=gen, device="cuda")).bfloat16()
    out, h = block.normed_prefill(x, res, gain, w, k, ranks=2)

    ry, rh = ox.add_rms_norm(down(x), down(gain), down(res))
    assert np.all(np.abs(down(h) - rh) <= 2.0 ** -8 * np.abs(rh) + 2.0 ** -24 * (np.abs(down(x)) + np.abs(down(res))))
    y = moe.moe_add_rms_norm(x, gain, res)[0]
    weight, expert, _ = moe.moe_gating_top_k(y @ w["router"].t(), k, bias=w["bias"], **block.ROUTING)
    weight, expert = down(weight), expert.cpu().numpy()
    xv = oe.mx_values(*oe.mx_quantize(ry))
    v13 = oe.mx_values(w["w13"].cpu().numpy(), w["s13"].cpu().numpy())
    v2 = oe.mx_values(w["w2"].cpu().numpy(), w["s2"].cpu().numpy())
    ref = np.zeros((T, H))
    for e in range(E):
        t, j = np.nonzero(expert == e)
        act = oe.mx_values(*oe.mx_quantize(oe.gated(xv[t], v13[e], I)[0]))
        ref[t] += (act @ v2[e].T) * weight[t, j][:, None]
    assert np.linalg.norm(down(out) - ref) <= 2.0 ** -8 * np.linalg.norm(ref)


@pytest.mark.parametrize("T", [37, 900])
def test_training_block_gradients(T):
    """examples/moe_training.py in float32 against torch's own gradients of the same formulas in float64, given the GPU's
    choice of experts.  A gradient passes six steps or fewer, each within 50 * 2^-24 of the size of its terms, and its terms
    cancel to no less than a quarter in norm: 2^-13 of its norm."""
    import torch

    block = example("moe_training")
    gen = torch.Generator(device="cuda").manual_seed(T)
    E, H, I, k = 6, 96, 64, 3
    p = block.parameters(E, H, I, gen, torch.float32)
    x, res, gy, gh = (torch.randn(T, H, generator=gen, device="cuda") for _ in range(4))
    x.requires_grad_()
    res.requires_grad_()
    y, h = block.block(x, res, p, k)
    torch.autograd.backward([y, h], [gy, gh])

    q = {n: v.detach().double().requires_grad_() for n, v in p.items()}
    a, b = (t.detach().double().requires_grad_() for t in (x, res))
    s = a + b
    z = s * torch.rsqrt(s.square().mean(1, keepdim=True) + 1e-6) * q["gain"]
    logits = z @ q["router"].t()
    expert = moe.moe_gating_top_k(logits.detach().float(), k, **block.ROUTING)[1].long()
    score = torch.sigmoid(logits).gather(1, expert)
    weight = score / score.sum(1, keepdim=True) * 2.5
    out = torch.zeros_like(z)
    for j in range(k):
        w13, w2 = q["w13"][expert[:, j]], q["w2"][expert[:, j]]
        g, u = torch.einsum("tih,th->ti", w13, z).chunk(2, -1)
        out = out + weight[:, j:j + 1] * torch.einsum("thi,ti->th", w2, torch.nn.functional.silu(g) * u)
    torch.autograd.backward([out, s], [gy.double(), gh.double()])
    near = lambda got, want: float((got.double() - want).norm()) <= 2.0 ** -13 * float(want.norm())  # noqa: E731
    assert near(y.detach(), out.detach()) and near(h.detach(), s.detach())
    assert near(x.grad, a.grad) and torch.equal(x.grad, res.grad)
    for n in p:
        assert near(p[n].grad, q[n].grad), n


def test_training_example_runs():
    example("moe_training").main()


def test_block_example_runs():
    example("moe_block").main()


def test_sorted_rows_through_the_grouped_product():
    """Quantised rows sorted by expert go straight into the experts' product, with counts and weights as they come, and an
    expert-parallel rank's share of the experts gives its share of the sum."""
    import torch

    rng = np.random.default_rng(0)
    T, E, H, N, k = 300, 6, 128, 64, 2
    x = torch.from_numpy(rng.standard_normal((T, H))).float().cuda()
    gain = torch.ones(H, device="cuda")
    w = torch.from_numpy(rng.standard_normal((E, N, H)) * H ** -0.5).float().cuda()
    wq, ws = moe.moe_mx_quantize(w)
    expert = torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(T)])).int().cuda()
    weight = torch.rand(T, k, device="cuda")
    _, _, q, s = moe.moe_add_rms_norm(x, gain, quant="mxfp4", return_y=False)
    total = torch.zeros(T, N, device="cuda")
    for first in (0, 4):                                            # two ranks: experts 0..3, and 4 and 5
        held = min(4, E - first)
        rows, scales, _, row_idx, num, row_weight = moe.moe_sort_tokens(q, expert, held, first_expert=first,
                                                                        per_token_scales=s, expert_topk_weight=weight)
        used = int(num.sum())
        y = moe.moe_mx_grouped_matmul(rows[:used].contiguous(), scales[:used].contiguous(), num, wq[first:first + held].contiguous(),
                                      ws[first:first + held].contiguous(), out_dtype=torch.float32,
                                      row_weight=row_weight[:used].contiguous(), check_status=True)
        total += moe.moe_combine_tokens(y, row_idx)
    values = oe.mx_values(q.cpu().numpy(), s.cpu().numpy())
    wv = oe.mx_values(wq.cpu().numpy(), ws.cpu().numpy())
    ref, size = np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        for j in range(k):
            e = int(expert[t, j])
            ref[t] += float(weight[t, j]) * (wv[e] @ values[t])
            size[t] += float(weight[t, j]) * np.sqrt((wv[e] ** 2) @ (values[t] ** 2))
    # the product's bound on its float32 sums (oracle.experts.sum_error), and a product and a sum or two of 2^-24 behind it
    bound = oe.sum_error(H, size ** 2) + 2.0 ** -21 * (size + np.abs(ref))
    assert np.all(np.abs(down(total) - ref) <= bound)
