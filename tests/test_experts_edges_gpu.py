"""Calls of the expert operators at the edges of what their headers allow, against the float64 oracle.

The tolerances are those of test_experts_gpu.py: the oracle's bound on float32 sums, h's 16-bit
roundings in the layer, and the result's own rounding.
"""
import ctypes
import time

import numpy as np
import pytest

import moe_expert_token_gb300 as moe
import moe_expert_token_gb300.mrr_v2 as m
from oracle import experts as ox
from test_experts_gpu import H_UNIT, UNIT, close, down, grouped_case, up, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from moe_expert_token_gb300 import build

    build.build()
    m.load_library()


def offset(a, n):
    """The device tensor of a numpy array, n elements past the start of an allocation."""
    import torch

    t = torch.from_numpy(np.ascontiguousarray(a))
    flat = torch.zeros(t.numel() + n, dtype=t.dtype, device="cuda")
    flat[n:] = t.reshape(-1).cuda()
    return flat[n:].view(t.shape)


def biased_layer(x, H, E, w13, s13, w2, s2):
    """A layer whose bias gives every token experts E - 1 and 1, with weights 3.5 / 5 and 1.5 / 5."""
    import torch

    wr = torch.zeros(E, H, dtype=torch.bfloat16, device="cuda")
    bias = torch.zeros(E, dtype=torch.bfloat16, device="cuda")
    bias[E - 1], bias[1] = 3.0, 1.0
    return moe.moe_few_token_layer(x, wr, w13, w2, 2, bias=bias, w13_scales=s13, w2_scales=s2, norm_type=1,
                                   check_status=True)


def biased_reference(x, E, v13, v2, h_unit):
    T = len(x)
    return ox.layer(x, np.tile(np.array([3.5, 1.5]) / 5.0, (T, 1)), np.tile([E - 1, 1], (T, 1)), np.full(T, 1e-6), v13,
                    v2, h_unit)


# ----------------------------------------------------------------------------- the unused scale byte of a last pair

@pytest.mark.parametrize("T", [1, 3, 7, 20])
@pytest.mark.parametrize("H,I", [(160, 96), (224, 224), (194, 222), (992, 736), (1026, 542)])
@pytest.mark.parametrize("off", [0, 2])
def test_layer_ignores_the_unused_scale_byte(T, H, I, off):
    """K mod 64 in 2, 30 and 32: the last pair's second byte stands for no block, and 255 (NaN) in it
    changes nothing.  Scale rows of 8-byte multiples and others, aligned and not."""
    import torch

    rng = np.random.default_rng(H + I + T)
    E = 3
    (w13, s13, v13), (w2, s2, v2) = weights(rng, E, 2 * I, H), weights(rng, E, H, I)
    s13[..., -1, 1] = s2[..., -1, 1] = 255
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16).cuda()
    y = biased_layer(x, H, E, up(w13), offset(s13, off), up(w2), offset(s2, off))
    ref, bound = biased_reference(down(x), E, v13, v2, (H_UNIT if T <= 4 else UNIT)["float16"])
    close(y, ref, bound, "bfloat16")


@pytest.mark.parametrize("K", [32, 96, 160, 224, 992])
def test_grouped_ignores_the_unused_scale_byte(K):
    def edit(s):
        s[..., -1, 1] = 255

    got, ref, bound = grouped_case(K, [3, 0, 40, 130], K, 48, out="float32", x_edit=edit, w_edit=edit)
    assert np.isfinite(ref).all()
    close(got, ref, bound, "float32")


@pytest.mark.parametrize("K", [2, 30, 96, 1026])
def test_dequantize_ignores_the_unused_scale_byte(K):
    import torch

    q, s = ox.mx_quantize(np.random.default_rng(K).standard_normal((3, K)))
    s[:, -1, 1] = 255
    assert np.array_equal(down(moe.moe_mx_dequantize(up(q), up(s), torch.float32)), ox.mx_values(q, s))


# ----------------------------------------------------------------------------- scales of unlike alignment

@pytest.mark.parametrize("T", [1, 4, 8, 20])
@pytest.mark.parametrize("H,I", [(200, 256), (456, 200), (242, 480)])
@pytest.mark.parametrize("off13,off2", [(2, 0), (1, 0), (4, 8), (0, 2), (0, 3)])
def test_layer_scales_of_unlike_alignment(T, H, I, off13, off2):
    """w13_scales and w2_scales aligned differently, where scale rows are 8-byte multiples (H and I of 193 to
    256 and 449 to 512), half of a stage's lanes have no bytes to bring (I = 200, 256), and the last items have
    fewer than 16 rows."""
    import torch

    rng = np.random.default_rng(H + I + T)
    E = 3
    (w13, s13, v13), (w2, s2, v2) = weights(rng, E, 2 * I, H), weights(rng, E, H, I)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16).cuda()
    y = biased_layer(x, H, E, up(w13), offset(s13, off13), up(w2), offset(s2, off2))
    ref, bound = biased_reference(down(x), E, v13, v2, (H_UNIT if T <= 4 else UNIT)["float16"])
    close(y, ref, bound, "bfloat16")


# ----------------------------------------------------------------------------- waits that run out

def limited(name, more):
    """The library's internal form of a run function, whose waits have a limit of their own and may be short
    of an arrival: `more` are the argtypes behind the public function's."""
    lib = m.load_library()
    f = getattr(lib, name + "_waits")
    f.restype = ctypes.c_int
    f.argtypes = [*getattr(lib, name).argtypes, *more]
    return f


LIMIT_NS = 20_000_000       # far more than a launch takes, far less than a test may


@pytest.mark.parametrize("short_of", [1, 2, 3, 4], ids=["full_stage", "empty_stage", "full_sums", "empty_sums"])
@pytest.mark.parametrize("A,N,gated", [(64, 5120, 0), (64, 2560, 1), (1600, 5120, 0), (1600, 2560, 1)])
def test_grouped_wait_that_runs_out_is_reported(short_of, A, N, gated):
    """One arrival less than a kind of barrier expects: the call ends soon, with MRR_ERR_TIMEOUT, and the next
    one is right.  More tiles than blocks have sets of sums for, more steps than the ring has stages; tiles of one
    weight tile and of two."""
    import torch

    E, K = 8, 2560
    gen = torch.Generator(device="cuda").manual_seed(A + N)
    byte = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=gen, device="cuda", dtype=torch.uint8)  # noqa: E731
    q, s = byte(0, 256, A, K // 2), byte(120, 128, A, K // 64, 2)
    w, ws = byte(0, 256, E, N * (1 + gated), K // 2), byte(120, 128, E, N * (1 + gated), K // 64, 2)
    c = torch.full((E,), A // E, dtype=torch.int32, device="cuda")
    want = moe.moe_mx_grouped_matmul(q, s, c, w, ws, gated=bool(gated), check_status=True)
    y = torch.empty_like(want)
    space = torch.empty(moe.moe_mx_grouped_workspace(E), dtype=torch.uint8, device="cuda")
    run = limited("moe_mx_grouped_run", [ctypes.c_uint64, ctypes.c_int])

    def call(short):
        st = run(q.data_ptr(), s.data_ptr(), A, K, c.data_ptr(), 0, 1, E, w.data_ptr(), ws.data_ptr(), N, gated, None,
                 y.data_ptr(), 1, None, space.data_ptr(), space.numel(), None, LIMIT_NS, short)
        assert st == m.MRR_OK
        return m.mrr_v2_read_status(space.data_ptr(), space.numel(), None)

    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert call(short_of) == m.MRR_ERR_TIMEOUT
    assert time.perf_counter() - t0 < 1.0
    y.zero_()
    assert call(0) == m.MRR_OK
    assert torch.equal(y, want)


@pytest.mark.parametrize("T,which", [(3, 0), (3, 2), (3, 3), (7, 3), (20, 0), (20, 1), (20, 2), (20, 3)])
@pytest.mark.parametrize("H,I,mx", [(512, 256, False), (70, 38, False), (512, 256, True), (66, 166, True)])
def test_layer_wait_that_runs_out_is_reported(T, which, H, I, mx):
    """A grid-wide wait that expects a block more than there are, or (3) copies whose barriers expect an arrival
    more: the call ends soon, with MRR_ERR_TIMEOUT, and what follows on the same workspace is right: a replay of the same graph, whose first wait goes by the same
    tag, on other inputs, and a plain call."""
    import torch

    E, k = 8, 2
    gen = torch.Generator(device="cuda").manual_seed(T + H)
    rnd = lambda *s: (torch.randn(*s, generator=gen, device="cuda") * s[-1] ** -0.5).bfloat16()  # noqa: E731
    xs = [rnd(T, H) * H ** 0.5 for _ in range(4)]
    wr, w13, w2, s13, s2 = rnd(E, H), rnd(E, 2 * I, H), rnd(E, H, I), None, None
    if mx:
        (w13, s13), (w2, s2) = moe.moe_mx_quantize(w13), moe.moe_mx_quantize(w2)
    want = [moe.moe_few_token_layer(x, wr, w13, w2, k, w13_scales=s13, w2_scales=s2, check_status=True) for x in xs]
    x, y = torch.empty_like(xs[0]), torch.empty_like(xs[0])
    short_of = torch.zeros(1, dtype=torch.int32, device="cuda")
    space = torch.full((moe.moe_few_token_layer_workspace(T, H, E, I, k),), 0xA5, dtype=torch.uint8, device="cuda")
    run = limited("moe_few_token_layer_run", [ctypes.c_uint64, ctypes.c_void_p])
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st = run(ptr(x), 1, T, H, ptr(wr), E, None, ptr(w13), ptr(s13), ptr(w2), ptr(s2), 3 if mx else 1, I, k, 1, 1, 1.0,
                 1e-20, 0, 0, ptr(y), None, None, ptr(space), space.numel(), torch.cuda.current_stream().cuda_stream,
                 LIMIT_NS, ptr(short_of))
    assert st == m.MRR_OK

    def replay(i, short):
        x.copy_(xs[i])
        y.zero_()
        short_of.fill_(short)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        graph.replay()
        st = m.mrr_v2_read_status(ptr(space), space.numel(), torch.cuda.current_stream().cuda_stream)
        assert time.perf_counter() - t0 < 1.0
        return st

    assert replay(0, 0) == m.MRR_OK and torch.equal(y, want[0])
    for i in (1, 2):
        assert replay(i, 1 + which) == m.MRR_ERR_TIMEOUT
        assert replay(i + 1, 0) == m.MRR_OK
        assert torch.equal(y, want[i + 1])
    again = moe.moe_few_token_layer(xs[1], wr, w13, w2, k, w13_scales=s13, w2_scales=s2, workspace=space, check_status=True)
    assert torch.equal(again, want[1])


# ----------------------------------------------------------------------------- NaN and infinity in weights

def chosen_layer(choice, E, H, I, w13, s13, w2, s2, dt, seed=0):
    """A layer whose tokens choose the experts of `choice` [T, 2] (in this order, by logits of 12 and 8
    against about 0): (y, the oracle's routing of the same inputs)."""
    import torch

    rng = np.random.default_rng(seed)
    f = lambda a: torch.from_numpy(a).to(getattr(torch, dt))  # noqa: E731
    x = rng.standard_normal((len(choice), H))
    x[:, :E] = 0
    for t, (a, b) in enumerate(choice):
        x[t, a], x[t, b] = 1.5, 1.0
    wr = np.zeros((E, H))
    wr[np.arange(E), np.arange(E)] = 8.0
    x, wr = f(x), f(wr)
    y, w, idx = moe.moe_few_token_layer(x.cuda(), wr.cuda(), w13, w2, 2, w13_scales=s13, w2_scales=s2,
                                        return_routing=True, check_status=True)
    rw, ridx, sure, error = ox.routing(down(x), down(wr), 2)
    assert sure.all() and np.array_equal(idx.cpu().numpy(), ridx) and ridx.tolist() == [list(c) for c in choice]
    return y, down(x), rw, ridx, 3 * error + 1e-5


@pytest.mark.parametrize("T", [2, 4, 5, 8, 12])
@pytest.mark.parametrize("H,I", [(96, 64), (2080, 320), (70, 1100)])
@pytest.mark.parametrize("mx", [False, True])
def test_layer_weights_of_an_expert_reach_only_its_tokens(T, H, I, mx):
    """NaN in rows of an expert's weights is the result of the tokens that chose it, and of no other."""
    import torch

    rng = np.random.default_rng(T + H)
    E = 8
    choice = [(1, 6)] + [(3, 4) if t % 2 else (4, 7) for t in range(1, T)]
    if mx:
        (w13, s13, v13), (w2, s2, v2) = weights(rng, E, 2 * I, H), weights(rng, E, H, I)
        s2[1, 5, 0, 0] = s2[6, H - 1, -1, 0] = 255
        v2 = ox.mx_values(w2, s2)
        w13, s13, w2, s2 = (up(a) for a in (w13, s13, w2, s2))
    else:
        w13, w2 = (torch.from_numpy(rng.standard_normal(s) * s[-1] ** -0.5).to(torch.bfloat16).cuda()
                   for s in ((E, 2 * I, H), (E, H, I)))
        w2[1, 5, 3] = w2[6, H - 1, I - 1] = float("nan")
        s13, s2, v13, v2 = None, None, down(w13), down(w2)
    y, x, rw, ridx, werr = chosen_layer(choice, E, H, I, w13, s13, w2, s2, "bfloat16")
    ref, bound = ox.layer(x, rw, ridx, werr, v13, v2, (H_UNIT if T <= 4 else UNIT)["float16" if mx else "bfloat16"])
    assert np.isnan(ref[0]).sum() == 2 and np.isfinite(ref[1:]).all()
    close(y, ref, bound, "bfloat16")


@pytest.mark.parametrize("T", [1, 3, 6, 12])
@pytest.mark.parametrize("dt", ["bfloat16", "float16"])
def test_layer_an_infinite_weight_gives_infinity(T, dt):
    """An infinity in a weight of the down product makes that element of y infinite, with the sign of h: a
    second part of h, which may be zero or of the other sign, must not make it NaN."""
    import torch

    rng = np.random.default_rng(T)
    E, H, I = 8, 80, 48
    w13, w2 = (torch.from_numpy(rng.standard_normal(s) * s[-1] ** -0.5).to(getattr(torch, dt)).cuda()
               for s in ((E, 2 * I, H), (E, H, I)))
    w2[4, :, 7] = float("inf")
    w2[4, ::2, 7] = float("-inf")
    y, x, rw, ridx, werr = chosen_layer([(4, 7)] * T, E, H, I, w13, None, w2, None, dt)
    ref, bound = ox.layer(x, rw, ridx, werr, down(w13), down(w2), (H_UNIT if T <= 4 else UNIT)[dt])
    assert np.isinf(ref).all()
    close(y, ref, np.where(np.isfinite(bound), bound, 0), dt)


# ----------------------------------------------------------------------------- what a caller's workspace may be

def test_workspace_of_other_memory_is_refused():
    """A workspace in host memory, or one whose bytes are not one after another, is refused, and one that
    is too small or not aligned reported: none of them reaches the kernel."""
    import torch

    q = torch.zeros(8, 32, dtype=torch.uint8, device="cuda")
    s = torch.full((8, 1, 2), 127, dtype=torch.uint8, device="cuda")
    c = torch.tensor([4, 4], dtype=torch.int32, device="cuda")
    w, ws = torch.zeros(2, 6, 32, dtype=torch.uint8, device="cuda"), torch.zeros(2, 6, 1, 2, dtype=torch.uint8, device="cuda")
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    wr, w13, w2 = (torch.zeros(*n, dtype=torch.bfloat16, device="cuda") for n in ((4, 64), (4, 64, 64), (4, 64, 32)))
    good = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for bad, err in ((torch.empty(1 << 20, dtype=torch.uint8), ValueError), (good[::2], ValueError),
                     (good[:1].expand(1 << 20), ValueError), (good[:64], m.MrrError), (good[16:], m.MrrError)):
        with pytest.raises(err):
            moe.moe_mx_grouped_matmul(q, s, c, w, ws, workspace=bad)
        with pytest.raises(err):
            moe.moe_few_token_layer(x, wr, w13, w2, 2, workspace=bad)
    moe.moe_mx_grouped_matmul(q, s, c, w, ws, workspace=good, check_status=True)
    moe.moe_few_token_layer(x, wr, w13, w2, 2, workspace=good, check_status=True)


# ----------------------------------------------------------------------------- the choice of experts

SEPARATED = [(1, 8, 2, 256, 128, 0, 1, 1), (1, 64, 8, 512, 48, 1, 8, 4), (1, 1024, 64, 512, 32, 1, 1, 1), (1, 60, 6, 200, 72, 2, 4, 3),
             (3, 256, 8, 512, 32, 0, 8, 2), (8, 1024, 64, 512, 32, 1, 16, 8), (9, 96, 4, 256, 40, 2, 1, 1),
             (64, 1024, 64, 512, 32, 1, 1, 1), (64, 64, 64, 256, 40, 0, 1, 1), (40, 1024, 7, 256, 32, 0, 32, 8)]


def separated(T, E, H, seed):
    """x [T, H] and router weights [E, H] in bfloat16 whose logits spread over -3 .. 3, each token's in an
    order of its own."""
    import torch

    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16)
    z = np.stack([rng.permutation(np.linspace(-3, 3, E)) for _ in range(T)])
    return x, torch.from_numpy(np.linalg.lstsq(x.double().numpy(), z, rcond=None)[0].T.copy()).to(torch.bfloat16)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T,E,k,H,I,norm,groups,keep", SEPARATED)
def test_layer_experts_are_the_oracles(T, E, k, H, I, norm, groups, keep, mx):
    """The experts, their order and weights, and y, against the oracle's own routing, with logits far enough apart
    for it to be certain of every token's (one token of a step among them, and the largest tables)."""
    x, wr = separated(T, E, H, T + E + H + 1)
    kw = dict(norm_type=norm, group_count=groups, k_group=keep, group_select_mode=groups > 1, routed_scaling_factor=1.5)
    rw, ridx, sure, error = ox.routing(x.double().numpy(), wr.double().numpy(), k, **kw)
    assert sure.all()
    rng = np.random.default_rng(E)
    if mx:
        (w13, s13, v13), (w2, s2, v2) = weights(rng, E, 2 * I, H), weights(rng, E, H, I)
        w13, s13, w2, s2 = (up(a) for a in (w13, s13, w2, s2))
    else:
        w13, w2 = (up(rng.standard_normal(s) * s[-1] ** -0.5, "bfloat16") for s in ((E, 2 * I, H), (E, H, I)))
        s13, s2, v13, v2 = None, None, down(w13), down(w2)
    y, w, idx = moe.moe_few_token_layer(x.cuda(), wr.cuda(), w13, w2, k, w13_scales=s13, w2_scales=s2,
                                        return_routing=True, check_status=True, **kw)
    assert np.array_equal(idx.cpu().numpy(), ridx)
    werr = 3 * error + 1e-5      # as in layer_case of test_experts_gpu.py
    assert np.all(np.abs(down(w) - rw) <= werr[:, None] * np.abs(rw) + 1e-9)
    ref, bound = ox.layer(x.double().numpy(), rw, ridx, werr, v13, v2,
                          (H_UNIT if T <= 4 else UNIT)["float16" if mx else "bfloat16"])
    close(y, ref, bound, "bfloat16")


# ----------------------------------------------------------------------------- precision between the products

@pytest.mark.parametrize("T,E,k,H,I", [(2, 8, 2, 512, 256), (5, 16, 4, 512, 256), (8, 12, 3, 1030, 90), (9, 16, 4, 512, 320),
                                       (33, 40, 5, 454, 200), (64, 8, 4, 512, 192), (64, 8, 4, 390, 70), (20, 40, 4, 96, 1040)])
@pytest.mark.parametrize("dt", ["bfloat16", "float16"])
@pytest.mark.parametrize("mx", [False, True])
def test_layer_error_is_that_of_rounding_once(T, E, k, H, I, dt, mx):
    """y's error against 64 bits is that of rounding the exact y once, whatever h is held in between the
    products: as two 16-bit parts its error does not show (2^-17 and less), and as one float16 part under a bfloat16 y
    it adds in squares an eighth of y's own: a factor of (1 + 1/64)^(1/2) = 1.008.  Float32 sums add 2^-20."""
    import torch

    rng = np.random.default_rng(T + H)
    f = lambda a: torch.from_numpy(a).to(getattr(torch, dt)).cuda()  # noqa: E731
    x, wr = f(rng.standard_normal((T, H))), f(rng.standard_normal((E, H)) * H ** -0.5)
    if mx:
        (w13, s13, v13), (w2, s2, v2) = weights(rng, E, 2 * I, H), weights(rng, E, H, I)
        w13, s13, w2, s2 = (up(a) for a in (w13, s13, w2, s2))
    else:
        w13, w2 = f(rng.standard_normal((E, 2 * I, H)) * H ** -0.5), f(rng.standard_normal((E, H, I)) * I ** -0.5)
        s13, s2, v13, v2 = None, None, down(w13), down(w2)
    y, w, idx = moe.moe_few_token_layer(x, wr, w13, w2, k, w13_scales=s13, w2_scales=s2, norm_type=1,
                                        return_routing=True, check_status=True)
    ref, _ = ox.layer(down(x), down(w), idx.cpu().numpy(), np.zeros(T), v13, v2, 0.0)
    once = torch.from_numpy(ref).to(getattr(torch, dt)).double().numpy()
    assert np.linalg.norm(down(y) - ref) <= 1.02 * np.linalg.norm(once - ref)


def test_a_second_copy_of_the_library_runs(tmp_path):
    import shutil

    import torch

    from moe_expert_token_gb300 import build

    path = str(tmp_path / "copy.so")
    shutil.copy(build.LIB_PATH, path)
    libs = [m.load_library(), m.load_library(path)]
    gen = torch.Generator(device="cuda").manual_seed(3)
    T, E, H, I, k = 3, 4, 64, 32, 2
    x, wr, w13, w2 = (torch.randn(*s, generator=gen, device="cuda").bfloat16() for s in ((T, H), (E, H), (E, 2 * I, H), (E, H, I)))
    ys = []
    for lib in libs:
        y, space = torch.empty_like(x), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        assert lib.moe_few_token_layer_run(
            x.data_ptr(), 1, T, H, wr.data_ptr(), E, None, w13.data_ptr(), None, w2.data_ptr(), None, 1, I, k, 1, 1, 1.0,
            1e-20, 0, 0, y.data_ptr(), None, None, space.data_ptr(), space.numel(), None) == m.MRR_OK
        torch.cuda.synchronize()
        ys.append(y)
    assert torch.equal(*ys)
