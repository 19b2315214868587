"""The example layer: every stage of a step against its 64-bit definition on what the stage
before left in the layer's buffers; both orders of the experts' rows give the same bits."""
import os
import sys

import numpy as np
import pytest
import torch

from gpu_util import note
from layer_util import NORM_DELTA, SILU_DELTA, check_rows, f64
from oracle import layer as ol

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

SMALL = dict(hidden=256, inner=128, experts=16, top_k=3, groups=4, top_groups=2, max_tokens=200)


def tokens(layer, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, layer.hidden, device="cuda", generator=g).to(torch.bfloat16)


def products(got, a, sa, x, experts):
    """As in the experts' own tests: one rounding to bf16, what the 8-bit MFMA cuts off, fp32 sums."""
    want, S, G = ol.experts_f8(f64(a), f64(sa), x.codes.double().numpy(), x.scale, experts)
    bound = np.abs(want) * 2.0 ** -8 + G * 7 * 2.0 ** -13 + S * (16 + 3 + x.K // 128) * 2.0 ** -24
    assert (np.abs(f64(got) - want) <= bound).all()


@pytest.mark.parametrize("T", [1, 2, 21, 22, 200])
def test_stages_of_a_step(T):
    from routed_layer import RoutedLayer
    note(f"routed layer T={T}")
    layer = RoutedLayer(**SMALL)
    k, P = layer.top_k, T * layer.top_k
    x, r = tokens(layer, T, 1), tokens(layer, T, 2)
    h = f64(x) + f64(r)
    got = layer.step(x, r)
    torch.cuda.synchronize()
    eps = float(np.float32(1e-6))
    _, y = ol.rms_norm(h, None, f64(layer.weight), eps)
    bytes_of = lambda t: t.reshape(-1).view(torch.uint8)  # noqa: E731
    assert (np.abs(f64(r) - h) <= np.abs(h) * (2.0 ** -8 + 2.0 ** -23)).all()
    assert (np.abs(f64(layer.y[:T]) - y) <= np.abs(y) * (2.0 ** -8 + 2 * NORM_DELTA)).all()
    _, y = ol.rms_norm(f64(r), None, f64(layer.weight), eps)
    a, sa = layer.a[:T], layer.sa[:T]
    check_rows("f8_block", "bf16", y, NORM_DELTA, bytes_of(a), bytes_of(sa), a.numel(), 4 * sa.numel())
    ids, w = ol.route(f64(layer.logits[:T]), f64(layer.bias), k, True, True, 4, 2, 2, 2.5)
    np.testing.assert_array_equal(layer.ids[:T].cpu().numpy(), ids)
    assert (np.abs(f64(layer.weights[:T]) - w) <= np.abs(w) * (2.0 ** -24 + 2.0 ** -43)).all()
    pair = torch.arange(P, device="cuda") // k
    products(layer.gate_up[:P], a[pair], sa[pair], layer.up, ids.reshape(-1))
    hh, sh = layer.h[:P], layer.sh[:P]
    check_rows("f8_block", "bf16", ol.silu_mul(f64(layer.gate_up[:P])), SILU_DELTA, bytes_of(hh), bytes_of(sh), hh.numel(), 4 * sh.numel())
    products(layer.answers[:P], hh, sh, layer.down, ids.reshape(-1))
    want, S = ol.combine(f64(layer.answers[:P]), f64(layer.weights[:T]), None, np.arange(P).reshape(T, k))
    assert (np.abs(f64(got) - want) <= np.abs(want) * 2.0 ** -8 + S * (2 * k + 2) * 2.0 ** -24).all()


def test_sorted_by_expert_gives_the_same_bits():
    from routed_layer import RoutedLayer
    one, two = RoutedLayer(**SMALL), RoutedLayer(**SMALL, grouped=True)
    for T in (1, 21, 22, 200, 7):
        note(f"routed layer grouped T={T}")
        x, r = tokens(one, T, T), tokens(one, T, T + 1)
        q = r.clone()
        assert torch.equal(one.step(x, r), two.step(x, q)) and torch.equal(r, q)
        assert torch.equal(one.ids[:T], two.ids[:T])


@pytest.mark.parametrize("grouped", [False, True])
def test_a_captured_step(grouped):
    """Replayed with new rows in its inputs, between eager steps of the same layer."""
    from routed_layer import RoutedLayer
    note(f"routed layer captured grouped={grouped}")
    layer = RoutedLayer(**SMALL, grouped=grouped)
    x, r = tokens(layer, 90, 1), tokens(layer, 90, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(x, r)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = layer.step(x, r)
    for i in range(3):
        a, b = tokens(layer, 90, 10 + i), tokens(layer, 90, 20 + i)
        x.copy_(a)
        r.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        kept, sums = out.clone(), r.clone()
        want = layer.step(a, b)
        torch.cuda.synchronize()
        assert torch.equal(kept, want) and torch.equal(sums, b)


def test_main_runs(capsys):
    import routed_layer
    note("routed layer main")
    routed_layer.main()
    assert "step 3" in capsys.readouterr().out
