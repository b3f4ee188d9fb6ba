"""Gradients that medusa_rope records: the transposed turn, against the float64 definition and
against differences; without grad the call is what it was."""
import numpy as np
import pytest

from oracle import paged as ref
from tests.helpers import bf16_to_f64, to_dev, to_host
from tests.paged import HALF, U, dev_ints, values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mg():
    import medusa_head_speculative_heads_gb300 as m
    m.build()
    return m


def host64(t):
    a = to_host(t.detach())
    return bf16_to_f64(a) if a.dtype == np.uint16 else a.astype(np.float64)


def leaf(a):
    return to_dev(a).requires_grad_()


def near(got, want, x, m, dtype):
    """8 u m (|x0| + |x1|) + half a step, by the largest element."""
    return np.all(np.abs(host64(got) - want) <= 16 * U * m * np.abs(ref.f64(x)).max() + HALF[dtype] * np.abs(want) + 1e-30)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("needs", [(1, 1), (1, 0), (0, 1), (1, None)], ids=str)
def test_gradients_of_both_inputs(mg, dtype, inter, needs):
    rng = np.random.default_rng(7)
    nl, T, d, r, m = 2, 9, 32, 20, 1.25
    spec, f, pos = mg.RopeSpec(r, interleaved=inter, magnitude=m), ref.rope_frequencies(r), np.arange(40, 40 + T)
    x = [values(rng, (nl, T, h, d), dtype) for h in (4, 2)]
    w = [values(rng, (nl, T, h, d), dtype) for h in (4, 2)]
    n = 1 if needs[1] is None else 2
    t = [leaf(a) if need else to_dev(a) for a, need in zip(x[:n], needs)] + [None] * (2 - n)
    for inverse in (False, True):
        plain = mg.medusa_rope(*(None if a is None else a.detach() for a in t), dev_ints(pos), spec, inverse=inverse)
        outs = mg.medusa_rope(*t, dev_ints(pos), spec, inverse=inverse)
        assert outs[1] is None if n == 1 else True
        for o, p, need in zip(outs[:n], plain, needs):
            assert torch.equal(o, p) and o.requires_grad == bool(need)
        some = [i for i in range(n) if needs[i]]
        grads = torch.autograd.grad([outs[i] for i in some], [t[i] for i in some], [to_dev(w[i]) for i in some])
        for i, g in zip(some, grads):
            assert near(g, ref.rope(w[i], pos, f, inter, m, not inverse), w[i], m, dtype)


def test_against_differences_and_twice(mg):
    """f = sum w rope(x)^2 / 2 is quadratic: a central difference is exact but for rounding."""
    rng = np.random.default_rng(8)
    spec, pos = mg.RopeSpec(8, magnitude=1.5), dev_ints([3, 70000])
    x, w, v = (values(rng, (1, 2, 1, 12), "f32") for _ in range(3))
    f = lambda t: (to_dev(w) * mg.medusa_rope(t, None, pos, spec)[0].square()).sum() / 2  # noqa: E731
    t = leaf(x)
    grad, = torch.autograd.grad(f(t), t, create_graph=True)
    twice, = torch.autograd.grad((grad * to_dev(v)).sum(), t)
    size = 1.5 ** 2 * np.abs(w).sum() * max(np.abs(x).max(), np.abs(v).max(), 2.0) ** 2
    for tok, e in ((0, 0), (0, 5), (1, 3), (1, 11)):
        up, down = x.copy(), x.copy()
        up[0, tok, 0, e] += 1.0
        down[0, tok, 0, e] -= 1.0
        assert abs((f(to_dev(up)) - f(to_dev(down))).item() / 2 - grad[0, tok, 0, e].item()) < 256 * U * size
        diff = torch.autograd.grad(f(a := leaf(up)), a)[0] - torch.autograd.grad(f(b := leaf(down)), b)[0]
        assert abs((diff.detach() * to_dev(v)).sum().item() / 2 - twice[0, tok, 0, e].item()) < 256 * U * size


def test_slices_broadcast_gradients_one_output_and_another_stream(mg):
    rng = np.random.default_rng(9)
    T, d = 700, 16
    spec, f, pos = mg.RopeSpec(d), ref.rope_frequencies(d), np.arange(T)
    qkv = leaf(values(rng, (1, T, 3, d), "f32"))
    q, k = qkv[:, :, :2], qkv[:, :, 2:]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    qo, ko = mg.medusa_rope(q, k, dev_ints(pos), spec, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    g, = torch.autograd.grad(ko.sum(), qkv)  # ones, all in one place; nothing for q
    torch.cuda.synchronize()
    want = ref.rope(np.ones((1, T, 1, d), np.float32), pos, f, inverse=True)
    assert torch.all(g[:, :, :2] == 0) and near(g[:, :, 2:], want, np.ones(1, np.float32), 1.0, "f32")
    qkv.grad = None
    mg.medusa_rope(q, None, dev_ints(pos), spec)[0].transpose(1, 2).contiguous().sum().backward()
    assert near(qkv.grad[:, :, :2], np.broadcast_to(want, (1, T, 2, d)), np.ones(1, np.float32), 1.0, "f32") and torch.all(qkv.grad[:, :, 2:] == 0)


def test_where_nothing_is_recorded(mg):
    rng = np.random.default_rng(10)
    spec, pos = mg.RopeSpec(32), dev_ints(np.arange(5))
    q = leaf(values(rng, (1, 5, 2, 32), "bf16"))
    want = mg.medusa_rope(q.detach(), None, pos, spec)[0]
    assert not want.requires_grad
    with torch.no_grad():
        assert not mg.medusa_rope(q, None, pos, spec)[0].requires_grad
    out = torch.empty_like(want)
    got, _ = mg.medusa_rope(q, None, pos, spec, q_out=out)
    assert got is out and not out.requires_grad and torch.equal(out, want)


def test_positions_changed_before_the_backward_pass_are_an_error(mg):
    q, pos = leaf(values(np.random.default_rng(11), (1, 5, 2, 32), "f32")), dev_ints(np.arange(5))
    out, _ = mg.medusa_rope(q, None, pos, mg.RopeSpec(32))
    pos += 1
    with pytest.raises(RuntimeError, match="modified"):
        out.sum().backward()


def test_a_captured_step_with_its_gradient(mg):
    rng = np.random.default_rng(12)
    spec, pos = mg.RopeSpec(64), dev_ints(np.arange(30))
    x = values(rng, (1, 30, 4, 64), "f32")
    t, w = leaf(x), to_dev(values(rng, (1, 30, 4, 64), "f32"))
    step = lambda: torch.autograd.grad((w * mg.medusa_rope(t, None, pos, spec)[0]).sum(), t)[0]  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    w.copy_(w * 2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, mg.medusa_rope(w, None, pos, spec, inverse=True)[0])
