"""Host-side refusals of the 4-bit linear layer, the logits call and the counting calls.  Made-up device
addresses: only where no GPU could be launched on them."""
import ctypes

import pytest

import medusa_head_speculative_heads_gb300 as mg
from medusa_head_speculative_heads_gb300 import binding as B_

torch = pytest.importorskip("torch")
if torch.cuda.is_available():
    pytest.skip("made-up device addresses", allow_module_level=True)

INVALID, ALIAS, WORKSPACE = 1, 3, 5


@pytest.fixture(scope="module", autouse=True)
def built():
    mg.build()


def at(n):
    return (n + 1) << 32


def linear(**o):
    a = dict(x=at(0), ldx=512, q=at(1), s=at(2), z=at(3), T=9, K=512, N=100, G=64, y=at(4), dt=1, st=None)
    a.update(o)
    return mg.lib().medusa_linear_w4(a["x"], a["ldx"], a["q"], a["s"], a["z"], a["T"], a["K"], a["N"], a["G"], a["y"], a["dt"], a["st"], None)


@pytest.mark.parametrize("o", [dict(x=None), dict(q=None), dict(s=None), dict(y=None), dict(T=-1), dict(K=0), dict(K=500), dict(N=0), dict(G=16), dict(G=256), dict(G=96, K=96 * 4),
                               dict(ldx=511), dict(ldx=516), dict(x=at(0) + 8), dict(q=at(1) + 4), dict(s=at(2) + 1), dict(y=at(4) + 1), dict(y=at(4) + 2, dt=0), dict(dt=2),
                               dict(T=0x7fffffff), dict(N=0x7fffffff), dict(K=0x7fffff80, ldx=0x7fffff80)])
def test_linear_refuses(o):
    assert linear(**o) == INVALID


@pytest.mark.parametrize("o", [dict(y=at(0)), dict(y=at(1) + 16), dict(y=at(2)), dict(y=at(3)), dict(y=at(4), st=at(4) + 8)])
def test_linear_refuses_overlaps(o):
    assert linear(**o) == ALIAS


def test_a_product_with_no_rows_launches_nothing():
    assert linear(T=0, x=None, y=None) == 0
    assert linear(T=0, K=33) == INVALID


def quantize(**o):
    a = dict(w=at(0), N=10, K=256, G=64, sym=0, dt=0, q=at(1), s=at(2), z=at(3))
    a.update(o)
    return mg.lib().medusa_w4_quantize(a["w"], a["N"], a["K"], a["G"], a["sym"], a["dt"], a["q"], a["s"], a["z"], None)


@pytest.mark.parametrize("o", [dict(w=None), dict(q=None), dict(s=None), dict(z=None), dict(N=0), dict(K=255), dict(G=48), dict(dt=4), dict(w=at(0) + 2), dict(q=at(1) + 2), dict(s=at(2) + 1)])
def test_quantize_refuses(o):
    assert quantize(**o) == INVALID


@pytest.mark.parametrize("o", [dict(q=at(0)), dict(s=at(0) + 64), dict(z=at(1)), dict(s=at(1) + 4), dict(z=at(2))])
def test_quantize_refuses_overlaps(o):
    assert quantize(**o) == ALIAS


def topology(n=7):
    return B_.medusa_dev_topology(n, 3, 2, 2, at(20), at(21), at(22), at(23))


def process(rules=None, **o):
    r = dict(counts=at(1), prompt_bits=at(2), repetition=at(3), frequency=at(4), presence=at(5), bias=at(6), mask=at(7), mask_row=at(8), bias_rows=1, n_masks=3)
    r.update(rules or {})
    a = dict(z=at(0), ld=1000, dt=1, tok=at(9), topo=topology(), B=2, N=7, V=1000, out=at(10), st=None)
    a.update(o)
    return mg.lib().medusa_logits_process(a["z"], a["ld"], a["dt"], ctypes.byref(B_.medusa_logits_rules(**r)), a["tok"], None if a["topo"] is None else ctypes.byref(a["topo"]),
                                          a["B"], a["N"], a["V"], a["out"], a["st"], None)


@pytest.mark.parametrize("o", [dict(z=None), dict(out=None), dict(dt=5), dict(B=0), dict(N=0), dict(V=0), dict(ld=999), dict(N=8), dict(tok=None), dict(z=at(0) + 1),
                               dict(z=at(0) + 2, dt=0), dict(out=at(10) + 2), dict(tok=at(9) + 1), dict(topo=topology(257), N=257), dict(V=0x7ffffff0, ld=0x7ffffff0), dict(st=at(11) + 2),
                               dict(topo=None, B=1 << 17, N=1 << 17)])
def test_process_refuses(o):
    assert process(**o) == INVALID


@pytest.mark.parametrize("r", [dict(bias_rows=3), dict(bias_rows=0), dict(n_masks=0), dict(mask_row=None), dict(counts=at(1) + 2), dict(mask=at(7) + 1), dict(repetition=at(3) + 2)])
def test_process_refuses_rules(r):
    assert process(rules=r) == INVALID


def test_process_refuses_overlaps():
    assert process(out=at(0)) == ALIAS  # bf16: not in place
    assert process(out=at(0), dt=0, ld=1004) == ALIAS and process(out=at(0) + 16, dt=0) == ALIAS
    for n in range(1, 10):
        assert process(out=at(n)) == ALIAS, n
    assert process(out=at(20)) == ALIAS and process(st=at(10)) == ALIAS


def count(**o):
    a = dict(tok=at(0), B=2, S=9, V=100, c=at(1), p=at(2), st=None)
    a.update(o)
    return mg.lib().medusa_count_tokens(a["tok"], a["B"], a["S"], a["V"], a["c"], a["p"], a["st"], None)


@pytest.mark.parametrize("o", [dict(tok=None), dict(B=0), dict(S=-1), dict(V=0), dict(c=None, p=None), dict(tok=at(0) + 1), dict(c=at(1) + 2), dict(p=at(2) + 3), dict(S=0x7fffffff), dict(V=0x7fffffff)])
def test_count_refuses(o):
    assert count(**o) == INVALID


def test_count_refuses_overlaps_and_takes_no_tokens():
    assert count(c=at(0)) == ALIAS and count(p=at(0) + 8) == ALIAS and count(p=at(1)) == ALIAS and count(st=at(1)) == ALIAS
    assert count(S=0, tok=None) == 0


def accepted(**o):
    a = dict(tok=at(0), path=at(1), acc=at(2), B=3, N=7, D=4, V=100, c=at(3), st=None)
    a.update(o)
    return mg.lib().medusa_count_accepted(a["tok"], a["path"], a["acc"], a["B"], a["N"], a["D"], a["V"], a["c"], a["st"], None)


@pytest.mark.parametrize("o", [dict(tok=None), dict(path=None), dict(acc=None), dict(c=None), dict(B=0), dict(N=0), dict(N=257), dict(D=-1), dict(D=17), dict(V=0), dict(path=at(1) + 1), dict(B=0x7fffffff)])
def test_accepted_refuses(o):
    assert accepted(**o) == INVALID


@pytest.mark.parametrize("o", [dict(c=at(0)), dict(c=at(1) + 4), dict(c=at(2)), dict(st=at(3) + 4)])
def test_accepted_refuses_overlaps(o):
    assert accepted(**o) == ALIAS


def test_the_binding_refuses_other_shapes_types_and_places():
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError, match="on a GPU"):
        mg.medusa_linear_w4(z(3, 64), z(5, 8, dt=i32), z(2, 5))
    with pytest.raises(TypeError):
        mg.medusa_linear_w4(z(3, 64, dt=torch.float16), z(5, 8, dt=i32), z(2, 5))
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        mg.medusa_linear_w4(z(3, 64), z(5, 8, dt=i32), z(2, 5), out_dtype=torch.float16)
    with pytest.raises(TypeError, match="must be a tensor"):
        mg.medusa_linear_w4(3, z(5, 8, dt=i32), z(2, 5))
    with pytest.raises(ValueError, match="on a GPU"):
        mg.medusa_w4_quantize(z(4, 64))
    with pytest.raises(TypeError):
        mg.medusa_w4_quantize(z(4, 64, dt=torch.float16))
    with pytest.raises(ValueError, match="on a GPU"):
        mg.medusa_logits_process(z(1, 2, 9, dt=f32))
    with pytest.raises(TypeError):
        mg.medusa_logits_process(z(1, 2, 9, dt=torch.float64))
    with pytest.raises(TypeError, match="Int"):
        mg.medusa_count_tokens(z(1, 2, dt=torch.int64), 9, counts=z(1, 9, dt=i32))
    with pytest.raises(ValueError, match="on a GPU"):
        mg.medusa_count_tokens(z(1, 2, dt=i32), 9, counts=z(1, 9, dt=i32))
    with pytest.raises(ValueError, match="on a GPU"):
        mg.medusa_count_accepted(z(1, 9, dt=i32), z(1, 2, dt=i32), z(1, 2, dt=i32), z(1, dt=i32))


def test_a_topology_of_another_device_is_refused():
    topo = B_.DevTopology(topology(), torch.zeros(1))
    with pytest.raises(ValueError, match="topo is on cpu, logits are on meta"):
        mg.medusa_logits_process(torch.zeros(2, 7, 10, device="meta"), tokens=torch.zeros(2, 7, dtype=torch.int32), topo=topo)
