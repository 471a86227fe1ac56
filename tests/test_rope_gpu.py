"""osm_rope and osm_rope_bwd on the GPU against a plain fp64 restatement."""
import numpy as np
import pytest
import torch

import cache_ref as ref
from online_softmax_tiled_attn_gb300 import binding

pytestmark = pytest.mark.gpu

# A result is a sum of two products with a cosine and a sine: the angle is off by 2^-25 half turns
# (9.4e-8), sine and cosine by 2 ulp (2^-23), the products and the sum by 2^-24 each, all relative
# to amplitude (|a| + |b|): 6e-7 together.  Then one rounding to the type.
ARITH = 6e-7
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def rand(shape, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


def tolerance(x, y, rot, layout, amplitude, dtype):
    m = np.zeros_like(x)
    i0 = np.arange(rot // 2) * (2 if layout == "interleaved" else 1)
    i1 = i0 + (1 if layout == "interleaved" else rot // 2)
    m[..., i0] = m[..., i1] = np.abs(x[..., i0]) + np.abs(x[..., i1])
    return HALF_STEP[dtype] * np.abs(y) * 1.001 + ARITH * abs(amplitude) * m


# B, H, N, d, rot
SHAPES = [(1, 1, 1, 64, 64), (2, 3, 7, 128, 128), (2, 5, 33, 64, 24), (1, 2, 130, 128, 32),
          (3, 8, 5, 96, 96), (2, 2, 3, 10, 6), (1, 1, 2, 2, 2), (1, 4, 600, 128, 64),
          (70, 32, 1, 128, 128), (2, 1, 4, 256, 208)]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,H,N,d,rot", SHAPES, ids=str)
def test_rope_and_its_adjoint(B, H, N, d, rot, dtype, layout):
    x = rand((B, N, H, d), 11 * N + d + rot, dtype)
    w = ref.rates(rot)
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(0, 100000, (B, N), generator=g, dtype=torch.int32)
    table = binding.rope_table(w)
    xt = x.cuda().transpose(1, 2)  # a projection's layout, read in place
    x64 = x.double().numpy().transpose(0, 2, 1, 3)
    for call, inverse, amp in ((binding.osm_rope, False, 1.0), (binding.osm_rope_bwd, True, 1.25)):
        y = call(xt, table, positions=pos.cuda(), layout=layout, amplitude=amp)
        want = ref.rotate(x64, pos.numpy(), w, layout, amp, inverse)
        err = np.abs(y.double().cpu().numpy() - want)
        assert np.all(err <= tolerance(x64, want, rot, layout, amp, dtype)), err.max()
        assert torch.equal(y[..., rot:].cpu(), x.transpose(1, 2)[..., rot:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions(layout):
    """Angles stay exact at the largest and at negative positions."""
    d = 128
    x = rand((1, 2, 6, d), 3, torch.float32)
    pos = torch.tensor([[0, 1, 1 << 24, 2 ** 31 - 1, -1, -2 ** 31]], dtype=torch.int32)
    w = ref.rates(d)
    y = binding.osm_rope(x.cuda(), binding.rope_table(w), positions=pos.cuda(), layout=layout)
    want = ref.rotate(x.double().numpy(), pos.numpy().astype(np.int64), w, layout)
    # the table's entries come from double rates over a double 2 pi: two roundings of 2^-53 of a
    # rate of at most one radian, times 2^31 positions
    tol = tolerance(x.double().numpy(), want, d, layout, 1.0, torch.float32) + \
        2.0 ** 31 * 2 * 2.0 ** -53 * 2 * np.abs(x.double().numpy()).max()
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= tol)


def test_default_positions_in_place_and_strided_output():
    B, H, N, d = 2, 4, 50, 64
    x = rand((B, H, N, d), 8, torch.bfloat16).cuda()
    table = binding.rope_table(binding.rope_rates(d))
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    want = binding.osm_rope(x, table, positions=pos)
    assert torch.equal(binding.osm_rope(x, table), want)
    assert torch.equal(binding.osm_rope(x, table, positions=pos.expand(B, N).contiguous()), want)
    wide = torch.full((B, N, H, 3 * d), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[..., d:2 * d].transpose(1, 2)  # the middle of each row
    binding.osm_rope(x, table, out=out)
    assert torch.equal(out, want)
    assert (wide[..., :d] == 7).all() and (wide[..., 2 * d:] == 7).all()
    same = binding.osm_rope(x, table, out=x)
    assert same is x and torch.equal(x, want)


def test_odd_offsets_give_the_same_values():
    """A row that starts off any vector boundary takes the general path, with the same result."""
    B, H, N, d = 2, 3, 9, 128
    base = rand((B, H, N, d + 3), 4, torch.bfloat16).cuda()
    x = base[..., 3:]
    table = binding.rope_table(binding.rope_rates(64))
    for layout in ("half", "interleaved"):
        a = binding.osm_rope(x, table, layout=layout)
        b = binding.osm_rope(x.contiguous(), table, layout=layout)
        assert torch.equal(a, b)


def test_adjoint_and_difference_quotient():
    """<R x, y> = <x, R* y>, and the backward pass matches differences of the forward one."""
    B, H, N, d = 2, 2, 17, 64
    table = binding.rope_table(binding.rope_rates(32))
    x, y = (rand((B, H, N, d), s, torch.float32).cuda() for s in (1, 2))
    fx = binding.osm_rope(x, table, layout="interleaved", amplitude=0.75)
    gy = binding.osm_rope_bwd(y, table, layout="interleaved", amplitude=0.75)
    a, b = (fx.double() * y.double()).sum().item(), (x.double() * gy.double()).sum().item()
    size = (fx.double().abs() * y.double().abs()).sum().item()
    assert abs(a - b) <= 4 * ARITH * size
    # linear: a step of 1 along one coordinate gives the gradient itself, to the roundings of two
    # forward results
    e = torch.zeros_like(x)
    for idx in ((0, 0, 3, 0), (1, 1, 16, 31), (0, 1, 5, 40)):
        e.zero_()
        e[idx] = 1.0
        f1 = binding.osm_rope(x + e, table, layout="interleaved", amplitude=0.75)
        quotient = ((f1.double() - fx.double()) * y.double()).sum().item()
        row = tuple(idx[:3])
        bound = 8 * ARITH * ((x[row].abs() + 1) * y[row].abs()).double().sum().item()
        assert abs(quotient - gy[idx].item()) <= bound


def test_graph_and_stream():
    """Captured into a graph and replayed on new inputs; issued on a side stream."""
    B, H, N, d = 1, 8, 64, 128
    x = rand((B, H, N, d), 9, torch.bfloat16).cuda()
    table = binding.rope_table(binding.rope_rates(d))
    out = torch.empty_like(x)
    want = binding.osm_rope(x, table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    binding.osm_rope(x, table, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.osm_rope(x, table, out=out)
    x2 = rand((B, H, N, d), 10, torch.bfloat16).cuda()
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, binding.osm_rope(x2, table))
