"""Expert routing and the experts' products on the GPU against plain 64-bit references, and a whole
layer (quantise, router product, route, experts) eager, on another stream and in a graph."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from decode_gemv_thinkbit_amd import qlinear as ql

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    ql.lib()
    return torch.device("cuda:0")


# ---------------------------------------------------------------- route
def check_route(logits, k, renormalize, dev):
    ids, weights = ql.moe_route(logits.to(dev), k, renormalize=renormalize)
    v = logits.double().numpy()
    want_ids, want = ref.route(v, k, renormalize)
    assert ids.dtype == torch.int32 and np.array_equal(ids.cpu().numpy(), want_ids)
    # exp of a difference rounded to half a step of its size, expf within 2 steps, a sum of at most E
    # terms and one division
    top = np.where(np.isfinite(v), v, 0.0).max(1, keepdims=True)
    spread = np.abs(np.where(np.isfinite(v), v, top) - top).max(1, keepdims=True)
    rel = (v.shape[1] + 8 + spread) * 2 * ref.EPS32
    assert (np.abs(weights.cpu().numpy() - want) <= rel * want + 2.0 ** -126).all()


@pytest.mark.parametrize("ty", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (5, 10, 3), (7, 65, 16), (33, 128, 8), (9, 129, 6), (3, 256, 1),
                                   (4, 300, 5), (2, 1024, 16), (130, 60, 4), (6, 16, 16)])
def test_route(dev, T, E, k, renormalize, ty):
    g = torch.Generator().manual_seed(T * E + k)
    logits = torch.randn(T, E, generator=g) * 2
    logits = logits.masked_fill(torch.rand(T, E, generator=g) < 0.1, -INF)
    if T > 2:
        logits[1] = -INF  # a padded token
    check_route(logits.to(ty), k, renormalize, dev)


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_ties_and_special_values(dev, renormalize):
    E, nan = 70, float("nan")
    rows = torch.zeros(9, E)
    rows[0] = 1.5                                       # all equal: ascending ids
    rows[1, ::2] = -0.0                                 # -0 and 0 are equal
    rows[2] = nan
    rows[2, 66] = -3.0                                  # one live expert
    rows[3] = nan
    rows[4, 5], rows[4, 69] = INF, INF                  # infinities share the weight
    rows[5] = torch.finfo(torch.float32).min            # the type's lowest value is still a logit
    rows[5, 3] = -INF
    rows[6] = -1e30
    rows[6, 68] = 0.0
    rows[7] = torch.arange(E).float() * 50              # weights that underflow
    rows[8] = torch.linspace(-1e-40, 1e-40, E)          # subnormal logits keep their order
    check_route(rows, 4, renormalize, dev)


def test_route_into_given_tensors(dev):
    logits = torch.randn(11, 40, device=dev)
    buf = torch.full((64 + 33 + 64,), -7, dtype=torch.int32, device=dev)
    ids = buf[64:97].view(11, 3)
    weights = torch.empty(11, 3, device=dev)
    got = ql.moe_route(logits, 3, ids=ids, weights=weights)
    assert got[0] is ids and got[1] is weights
    want = ql.moe_route(logits, 3)
    assert torch.equal(ids, want[0]) and torch.equal(weights, want[1])
    assert (buf[:64] == -7).all() and (buf[97:] == -7).all()


# ---------------------------------------------------------------- experts
def stacks(E, H, I, seed, dev):
    return (ref.random_mx4((E, I, H), seed, dev, 118, 122), ref.random_mx4((E, I, H), seed + 1, dev, 118, 122),
            ref.random_mx4((E, H, I), seed + 2, dev, 118, 122))


def inputs(T, H, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, generator=g) / 16).to(torch.bfloat16)


def check_moe(x, ids, weights, experts, dev):
    y = ql.mx4_moe(x.to(dev), ids.to(dev), weights.to(dev), *experts)
    want, bound = ref.moe(x.double().numpy(), ids.numpy(), weights.double().numpy(), *(ref.host(t) for t in experts))
    got = y.cpu().numpy().astype(np.float64)
    off = np.abs(got - want)
    assert (off <= bound + 1e-300).all(), float((off / (bound + 1e-300)).max())
    assert torch.equal(y, ql.mx4_moe(x.to(dev), ids.to(dev), weights.to(dev), *experts))  # deterministic
    return y


@pytest.mark.parametrize("T,E,k,H,I", [(1, 1, 1, 32, 32), (1, 8, 2, 256, 128), (2, 5, 3, 96, 160), (3, 64, 8, 512, 224),
                                       (7, 10, 3, 416, 352), (16, 4, 2, 128, 64), (17, 2, 1, 160, 96), (33, 6, 4, 288, 736),
                                       (64, 3, 2, 192, 128), (64, 130, 16, 64, 32), (5, 1024, 8, 32, 32)])
def test_moe(dev, T, E, k, H, I):
    g = torch.Generator().manual_seed(T + E)
    ids, weights = ref.route(torch.randn(T, E, generator=g).double().numpy(), k, True)
    check_moe(inputs(T, H, 5), torch.from_numpy(ids), torch.from_numpy(weights).float(), stacks(E, H, I, T, dev), dev)


@pytest.mark.parametrize("T,E,k,H,I", [(1, 3, 1, 32, 96), (1, 8, 5, 64, 1056), (1, 16, 16, 96, 288), (1, 20, 9, 64, 1024),
                                       (2, 8, 2, 64, 2080), (3, 4, 3, 96, 4128), (2, 3, 2, 64, 12320), (5, 3, 1, 32, 6176),
                                       (8, 40, 4, 2080, 96), (64, 16, 4, 2048, 32), (20, 6, 4, 64, 2048),
                                       (64, 130, 16, 1568, 64), (64, 2, 1, 96, 1056)])
def test_moe_shared_and_long_rows(dev, T, E, k, H, I):
    """One token's experts among several waves, long rows of the down projection in parts, long inputs."""
    g = torch.Generator().manual_seed(T + I)
    ids, weights = ref.route(torch.randn(T, E, generator=g).double().numpy(), k, True)
    check_moe(inputs(T, H, 6), torch.from_numpy(ids), torch.from_numpy(weights).float(), stacks(E, H, I, T, dev), dev)


@pytest.mark.parametrize("ids", [[3, -1, 3, 9, 0], [-1, -1, -1, -1, -1], [6, 6, 6, 6, 6], [-1, 2, 7, -9, 1]])
@pytest.mark.parametrize("I", [64, 1120])
def test_moe_one_token_dropped_and_repeated(dev, ids, I):
    ids = torch.tensor([ids], dtype=torch.int32)
    weights = torch.tensor([[0.5, 0.25, -1.5, 2.0, 0.75]])
    is_ = (ids >= 0) & (ids < 7)
    experts, x = stacks(7, 96, I, 9, dev), inputs(1, 96, 2)
    y = check_moe(x, ids, torch.where(is_, weights, 0.0), experts, dev)
    loud = torch.where(is_, weights, float("nan"))
    assert torch.equal(y, ql.mx4_moe(x.to(dev), ids.to(dev), loud.to(dev), *experts))


@pytest.mark.parametrize("T,I", [(1, 1120), (2, 2080)])
def test_moe_infinite_weight(dev, T, I):
    """A weight multiplies an expert's whole sum, also where its rows are shared out: infinities keep signs."""
    experts, x = stacks(4, 64, I, 2, dev), inputs(T, 64, 4).to(dev)
    ids = torch.tensor([[2, 1]] * T, dtype=torch.int32, device=dev)
    y = ql.mx4_moe(x, ids, torch.tensor([[1.0, 0.0]] * T, device=dev), *experts)
    z = ql.mx4_moe(x, ids, torch.tensor([[INF, 0.0]] * T, device=dev), *experts)
    assert (y != 0).all() and torch.equal(z, torch.where(y > 0, INF, -INF))


def test_moe_beyond_four_gigabytes(dev):
    """Experts whose codes lie beyond 32-bit offsets, and the same experts alone."""
    E, H, I = 68, 8192, 16384
    last = stacks(2, H, I, 3, dev)
    big = [ql.Mx4Tensor(torch.zeros(E, *t.codes.shape[1:], dtype=torch.uint8, device=dev),
                        torch.zeros(E, *t.scales.shape[1:], dtype=torch.uint8, device=dev)) for t in last]
    for b, t in zip(big, last):
        assert b.codes.numel() > 1 << 32
        b.codes[-2:] = t.codes
        b.scales[-2:] = t.scales
    for T in (1, 2):  # as many pairs as experts at least: laid out alike, so equal
        ids = torch.arange(T, device=dev, dtype=torch.int32).view(T, 1)
        x, w = inputs(T, H, 5).to(dev), torch.ones(T, 1, device=dev)
        y, z = ql.mx4_moe(x, ids + (E - 2), w, *big), ql.mx4_moe(x, ids, w, *last)
        assert torch.equal(y, z) and (z != 0).any()


def test_moe_all_tokens_one_expert(dev):
    T, E, H, I = 64, 9, 128, 96
    ids = torch.full((T, 1), 8, dtype=torch.int32)
    check_moe(inputs(T, H, 1), ids, torch.rand(T, 1), stacks(E, H, I, 4, dev), dev)


def test_moe_dropped_and_repeated_ids(dev):
    """Ids outside the experts are left out (a row of them gives zeros), the same expert may come twice."""
    T, E, H, I = 6, 7, 160, 128
    ids = torch.tensor([[0, 6, -1], [-1, -1, -1], [3, 3, 3], [7, 2, 1 << 30], [-(1 << 31), 5, 5], [0, 0, 6]],
                       dtype=torch.int32)
    weights = torch.tensor([[0.5, 0.25, INF], [INF, float("nan"), 1.0], [0.25, -0.5, 2.0], [1.0, 0.125, 3.0],
                            [9.0, 0.3, 0.6], [0.0, 1.0, 0.7]])
    clean = torch.where((ids >= 0) & (ids < E), weights, 0.0)
    experts = stacks(E, H, I, 9, dev)
    x = inputs(T, H, 2)
    y = check_moe(x, ids, clean, experts, dev)
    assert (y[1] == 0).all()
    assert torch.equal(y, ql.mx4_moe(x.to(dev), ids.to(dev), weights.to(dev), *experts))  # their weights are not read
    none = torch.full_like(ids, -1)
    assert (ql.mx4_moe(x.to(dev), none.to(dev), weights.to(dev), *experts) == 0).all()


def test_moe_nan_stays_with_its_tokens(dev):
    """A NaN scale in one expert reaches the tokens that chose it and no others."""
    T, E, H, I = 5, 6, 128, 64
    gate, up, down = stacks(E, H, I, 3, dev)
    up.scales[4, 10, 1] = 255
    ids = torch.tensor([[4, 0], [1, 2], [3, 4], [5, 0], [2, 1]], dtype=torch.int32, device=dev)
    y = ql.mx4_moe(inputs(T, H, 2).to(dev), ids, torch.ones(T, 2, device=dev), gate, up, down)
    assert torch.isnan(y[[0, 2]]).all() and torch.isfinite(y[[1, 3, 4]]).all()


def test_moe_guarded_buffers(dev):
    """Outputs inside larger buffers and a workspace of exactly its size: nothing beside them is written."""
    T, E, k, H, I = 9, 12, 3, 96, 64
    experts, x = stacks(E, H, I, 6, dev), inputs(T, H, 3).to(dev)
    ids, weights = ql.moe_route(torch.randn(T, E, device=dev), k)
    need = ql.lib().qlinear_mx4_moe_workspace_bytes(T, k, E, H, I)
    ws = torch.full((256 + need + 256,), 0x5A, dtype=torch.uint8, device=dev)
    buf = torch.full((64 + T * H + 64,), 7.0, device=dev)
    y = ql.mx4_moe(x, ids, weights, *experts, out=buf[64:64 + T * H].view(T, H), workspace=ws[256:256 + need])
    assert (buf[:64] == 7).all() and (buf[64 + T * H:] == 7).all()
    assert (ws[:256] == 0x5A).all() and (ws[256 + need:] == 0x5A).all()
    assert torch.equal(y, ql.mx4_moe(x, ids, weights, *experts))


# ---------------------------------------------------------------- together
class Layer:
    """A router and experts quantised from dense weights, as a program would hold them."""

    def __init__(self, T, E, k, H, I, dev):
        g = torch.Generator(device=dev).manual_seed(1)
        self.k = k
        self.dense = [torch.randn(*s, generator=g, device=dev) * 0.05 for s in ((E, I, H), (E, I, H), (E, H, I))]
        self.router = ql.mx4_quantize(torch.randn(E, H, generator=g, device=dev) * 0.05)
        self.experts = [ql.mx4_quantize(w) for w in self.dense]
        self.shared = ql.mx4_quantize(torch.randn(H, H, generator=g, device=dev) * 0.05)

    def __call__(self, x):
        logits = ql.mx4_gemv(x, self.router)
        ids, weights = ql.moe_route(logits, self.k)
        y = ql.mx4_moe(x, ids, weights, *self.experts)
        return y, ql.mx4_gemm(ql.mx4_quantize(x), self.shared), ids, weights


def test_layer_against_reference(dev):
    T, E, k, H, I = 12, 16, 4, 256, 160
    layer, x = Layer(T, E, k, H, I, dev), inputs(T, H, 8) * 16
    y, z, ids, weights = layer(x.to(dev))
    logits, _ = ref.product(x.double().numpy(), ref.host(layer.router))
    want_ids, want_weights = ref.route(logits, k, True)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    for t, w in zip(layer.experts, layer.dense):  # the experts are the quantised dense weights
        codes, scales = ref.quantize(w[:2].double().cpu().numpy())
        assert np.array_equal(t.codes[:2].cpu().numpy(), codes) and np.array_equal(t.scales[:2].cpu().numpy(), scales)
    want, bound = ref.moe(x.double().numpy(), want_ids, weights.double().cpu().numpy(), *map(ref.host, layer.experts))
    assert (np.abs(y.cpu().numpy() - want) <= bound).all()
    xq = ref.values(*ref.quantize(x.double().numpy()))
    want, bound = ref.product(xq, ref.host(layer.shared))
    assert (np.abs(z.cpu().numpy() - want) <= bound).all()


def test_layer_on_another_stream(dev):
    layer, x = Layer(4, 8, 2, 256, 128, dev), inputs(4, 256, 8).to(dev)
    want = layer(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [layer(x) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)


def test_two_layers_in_graphs(dev):
    """Two captured layers with memory of their own, replayed in turn with eager work between."""
    layers = [Layer(6, 8, 2, 256, 128, dev), Layer(6, 24, 5, 320, 96, dev)]
    xs = [torch.zeros(6, h, dtype=torch.bfloat16, device=dev) for h in (256, 320)]
    graphs, outs = [], []
    for layer, x in zip(layers, xs):
        layer(x)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer(x))
        graphs.append(g)
    for step in range(4):
        for i in (0, 1):
            xs[i].copy_(inputs(6, xs[i].shape[1], 20 + step))
            graphs[i].replay()
        eager = [layer(x) for layer, x in zip(layers, xs)]
        torch.cuda.synchronize()
        for got, want in zip(outs, eager):
            for a, b in zip(got, want):
                assert torch.equal(a, b), step


def test_layers_at_once_on_two_streams(dev):
    """Two layers under way together, each on a stream of its own, give what they give alone."""
    layers = [Layer(16, 16, 5, 512, 288, dev), Layer(2, 8, 2, 256, 2080, dev)]
    xs = [inputs(16, 512, 8).to(dev), inputs(2, 256, 9).to(dev)]
    want = [layer(x) for layer, x in zip(layers, xs)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(20):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(layers[i](xs[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for g in got[i]:
            for a, b in zip(g, want[i]):
                assert torch.equal(a, b)
